// Attention over a paged MX cache for few rows a key/value head (sm_103a):
// decoding, 8 or 16 rows a tile.
//
// Every byte of the cache is read once by the tile that needs it, so the
// kernel is meant to be bound by HBM: 8-bit heads of 128 bring an SM some 23
// values per clock, of which each costs 3.6 instructions of a lane here.  64 sequences to
// 4096 tokens, 32 heads of 128: 8 bits 233 us (87% of the measured copy rate),
// where 4 bits are bound by those instructions; one row over 1000 tokens 7.6 us,
// launch, lookups and one round; over 131072, 5 key heads, 4 bits 38.9.  A tensor-core
// tile of 128 rows would be empty but for 8, so the products are mma.sync's
// (m16n8k16, fp16 in, fp32 out), with the tokens or head values on M and the
// rows on N:
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
// Warps take groups of 16 tokens in turn (they lie in one page, a run each of
// K and V), by asynchronous copies into stages of their own, some 150 KB an SM
// under way; each keeps a maximum, sum and accumulator of its own.  They are
// joined in shared memory, and the CTAs of a cluster, which share a tile's
// keys, through distributed shared memory, in a fixed order.  Where even 8
// CTAs a tile leave SMs idle, several clusters share it, and a second kernel
// joins what they leave in the caller's workspace.
#include <cstdint>
#include <type_traits>

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
constexpr int kJoinThreads = kThreads;  // (few_plain has the same warps in both kernels)

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

// 16 bytes (4) to shared memory, there after cp_wait; with _if zeros where not `ok`.
__device__ __forceinline__ void cp_async16(uint32_t to, const uint8_t *from) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t to, const uint8_t *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async16_if(uint32_t to, const uint8_t *from, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4_if(uint32_t to, const uint8_t *from, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

template <int kWords>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[kWords]) {
    if constexpr (kWords >= 4) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(at + 4 * i)
                         : "memory");
    } else if constexpr (kWords == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    } else {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
    }
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t at) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}

// Where a warp's sums lie in shared memory.  Lanes (g, t) store two values of
// row 2t or 2t + 1 at a time, in the g-th of eight runs of the row: rows and
// runs all begin in the same banks, so pairs within a run are permuted by
// t and g, and 16 lanes meet in no bank (stored as they come they all did: one
// row over 1000 tokens 7.7 us, so 7.4; 64 sequences to 4096 234, so 229).
template <int kDP>
__device__ __forceinline__ int sum_swizzle(int r, int g) {
    return kDP == 128 ? (r >> 1 & 3) | (g >> 1 & 1) << 2 : r >> 1 & 3;
}
// The place of values d .. d + 3, pairs swapped where the permutation is odd.
template <int kDP>
__device__ __forceinline__ int sum_place(int r, int d) {
    constexpr int kRun = kDP / 8;
    const int g = d / kRun;
    return g * kRun + 4 * (d % kRun / 4 ^ sum_swizzle<kDP>(r, g) >> 1);
}

// Sums over parts of the keys, each under a maximum of its own.
struct Joined {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    __device__ __forceinline__ void add(float mi, float m, float li, float4 v) {
        // (A part without a maximum has zeros, or NaN where its scores are.)
        const float by = mi == -INFINITY ? 0.f : ex2(mi - m);
        l += mi == -INFINITY ? li : by * li;
        o.x = fmaf(by, v.x, o.x), o.y = fmaf(by, v.y, o.y), o.z = fmaf(by, v.z, o.z), o.w = fmaf(by, v.w, o.w);
    }
    // Four outputs from value d on.  A row that sees nothing has no sum: zeros.  One that does, and has none, has scores
    // of minus infinity alone, whose softmax is NaN.
    __device__ __forceinline__ void store(const MxAttentionArgs &a, const RowTile &tile, int row, int head, int group,
                                          int d, int nan_from) const {
        const long long at = (long long)(tile.start + row / group) * a.y_token +
                             (long long)(head * group + row % group) * a.y_head + d;
        const int sees = keys_of(tile, row, group, a.causal);
        const float by = nan_from < sees || (l == 0.f && sees > 0) ? __int_as_float(0x7FC00000) : l == 0.f ? 0.f : 1.f / l;
        store4(a.y, a.type, at, a.vec, make_float4(o.x * by, o.y * by, o.z * by, o.w * by));
    }
};

// kDP: the head's values rounded up to 64 or 128; kNR: row tiles of 8; kNP:
// fp16 terms of a query value and a probability.
template <int kBits, int kDP, int kNR, int kNP>
struct FewShared {
    static constexpr int kR = 8 * kNR;
    static constexpr int kPitch = kDP + 8;                   // halves of a staged query row
    static constexpr int kRow = kDP * kBits / 8;             // bytes of a staged token
    static constexpr int kStage = 32 * kRow + 128;           // K, V, and a scale word each
    static constexpr int kStages = kRow == 128 ? 3 : kRow == 64 ? 5 : 8;
    union {
        uint8_t stage[kFewWarps][kStages][kStage];
        float o[kFewWarps][kR][kDP];  // each warp's sums; the CTA's in [0]
    };
    __half q[kNP][kR][kPitch];
    uint2 mults[kFewWarps][32];  // of a token's blocks, K's of 16 tokens and V's
    float m[kFewWarps][kR], l[kFewWarps][kR];
    float m_all[kR], l_all[kR];
    int power[kR];    // of two, taken out of a query row
    int nan_from[4];  // first position whose v has NaN in a block
};

// Sums of one part of a tile's keys in the workspace: `parts` of these a tile,
// for each of its rows kDP outputs, then the maximum and the sum, and at the end nan_from.
__host__ __device__ constexpr size_t few_part_floats(int rows, int dp) { return (size_t)rows * (dp + 2) + 4; }

// Sums that are not to be used: M kSpoiltMax, so that they outweigh all others, and l kSpoilt.
constexpr float kSpoiltMax = 3e38f, kSpoilt = INFINITY;

struct PlainScratch {
    float o[kFewWarps][128], m[kFewWarps];
};

// The rows of tile and head `item` that CTA `rank` of S stores, kHere at once, by plain_row, the keys of a row
// shared by the warps.  (At the end of a kernel, and a function of its own that finds its tile anew: anywhere else, or
// with what it needs held for it, a CTA takes 0.2 us longer.)
template <int kBits, int kR, int kHere>
__device__ __noinline__ void few_plain(const MxAttentionArgs &a, int group, unsigned item, int rank, int S, PlainScratch &sh) {
    const RowTile tile = row_tile(a.batch, item / (unsigned)a.cache.heads, group, kR, a.tokens);
    const int head = (int)(item % (unsigned)a.cache.heads), lane = threadIdx.x & 31, warp = threadIdx.x / 32, d = 4 * lane;
    const int keys = min(keys_of(tile, tile.first + tile.rows - 1, group, a.causal), table_keys(a.batch.width, a.cache.page));
    for (int r = rank * kHere; r < tile.rows; r = (r + 1) % kHere ? r + 1 : r + 1 + (S - 1) * kHere) {
        const int row = tile.first + r;
        const PlainSums own = plain_row<kBits>(a, tile, row, group, head, keys, warp, 0x7FFFFFFF, kFewWarps);
        *reinterpret_cast<float4 *>(&sh.o[warp][d]) = own.o;
        if (lane == 0) sh.m[warp] = own.m;
        __syncthreads();
        if (warp == 0 && d < a.cache.D) {
            float top = -INFINITY, l = 0.f;
            for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, sh.m[w]);
            for (int w = 0; w < kFewWarps; ++w) l += ex2(sh.m[w] - (top == -INFINITY ? 0.f : top));
            const float none = l == 0.f && keys_of(tile, row, group, a.causal) > 0 ? __int_as_float(0x7FC00000) : 0.f;
            float4 y = make_float4(none, none, none, none);
            for (int w = 0; w < kFewWarps; ++w) {
                if (sh.m[w] == -INFINITY) continue;
                const float4 v = *reinterpret_cast<const float4 *>(&sh.o[w][d]);
                const float t = sh.m[w] - top - lg2(l), whole = floorf(t), by = ex2(t - whole);
                const int e = (int)fmaxf(whole, -999.f);
                y.x += scaled(v.x * by, e), y.y += scaled(v.y * by, e), y.z += scaled(v.z * by, e), y.w += scaled(v.w * by, e);
            }
            const long long at = (long long)(tile.start + row / group) * a.y_token +
                                 (long long)(head * group + row % group) * a.y_head + d;
            store4(a.y, a.type, at, a.vec, y);
        }
        __syncthreads();
    }
}

template <int kBits, int kDP, int kNR, int kNP>
__global__ void __launch_bounds__(kThreads, kNR == 1 && kNP == 1 ? 2 : 1)
    mx_attention_few_kernel(const __grid_constant__ MxAttentionArgs a, const int group, const int parts) {
    using Shared = FewShared<kBits, kDP, kNR, kNP>;
    constexpr int kR = Shared::kR, kRow = Shared::kRow, kStages = Shared::kStages;
    constexpr int kSteps = kDP / 16;                 // of 16 head values
    constexpr int kKRun = kDP / 4, kVRun = kDP / 8;  // neighbouring values of a lane
    constexpr int kKW = kKRun * kBits / 32, kVW = kVRun * kBits / 32;
    constexpr int kLanes = kRow / 16, kEach = 32 / kLanes;  // 16-byte pieces of a token, tokens a copy
    extern __shared__ __align__(16) uint8_t raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), g = lane >> 2, t = lane & 3;
    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int D = a.cache.D, blocks = D / kMxBlock;

    pdl_wait();
    // (Divisions of 32 bits here and below: ones of 64 take a hundred instructions each.)
    unsigned item = blockIdx.x / (unsigned)S;
    const int part = (int)(item % (unsigned)parts);
    item /= (unsigned)parts;
    const int head = (int)(item % (unsigned)a.cache.heads);
    const RowTile tile = row_tile(a.batch, item / (unsigned)a.cache.heads, group, kR, a.tokens);
    if (tile.rows == 0) return;  // with the whole cluster

    // Keys that any row sees, in groups, and this CTA's share of them.
    int keys = keys_of(tile, tile.first + tile.rows - 1, group, a.causal);
    const int room = table_keys(a.batch.width, a.cache.page);
    if (keys > room) {
        if (threadIdx.x == 0) atomicOr(a.status, kStatusIndex);
        keys = room;
    }
    const int groups = (keys + kFewGroup - 1) / kFewGroup;
    const int share = part * S + rank, shares = parts * S;
    auto first_group = [&](int i) {
        return shares < 1024 && groups < 1 << 21 ? (int)((unsigned)groups * (unsigned)i / (unsigned)shares)
                                                 : (int)((long long)groups * i / shares);
    };
    const int g0 = first_group(share), g1 = first_group(share + 1);

    // The warp's query rows, on their way while the first page is looked up.
    constexpr int kEachLane = kDP / 32;
    std::conditional_t<kNP == 2, float, uint16_t> query[kNR][kEachLane];
    const bool narrow = kNP == 2 && a.type != MxType::kF32;  // 16-bit rows as fp32 ones
#pragma unroll
    for (int n = 0; n < kNR; ++n) {
        const int r = warp + kFewWarps * n, row = tile.first + r;
        const long long at = (long long)(tile.start + row / group) * a.q_token +
                             (long long)(head * group + row % group) * a.q_head + lane;
        const auto *x = static_cast<const std::remove_reference_t<decltype(query[0][0])> *>(a.q) + at;
#pragma unroll
        for (int i = 0; i < kEachLane; ++i) {
            query[n][i] = 0;
            if (r >= tile.rows || lane + 32 * i >= D) continue;
            if (narrow)
                query[n][i] = wide_value(a.q, a.type, at + 32 * i);
            else
                query[n][i] = x[32 * i];
        }
    }

    // The warp's groups, every kFewWarps-th: copies of the next ones under way.
    const int per_page = a.cache.page / kFewGroup, row_bytes = D * kBits / 8;
    int piece = (g0 + warp) / per_page, within = (g0 + warp) % per_page;  // page and group within it
    int ahead = g0 + warp;                                                // the next group to copy
    auto next_page = [&]() { return ahead < g1 ? page_of(a.batch, a.cache, tile.seq, piece, a.status) : -1; };
    int page = next_page();
    uint32_t bad = 0;  // a bit a stage: its group is in no page
    // A token's 16-byte pieces are staged in an order that depends on the
    // token, so that the fragments' loads meet in no bank (8 bits) or in two.
    const int c = lane % kLanes, tok0 = lane / kLanes;
    auto swizzle = [](int tok, int piece16) { return kRow == 128 ? piece16 ^ (tok & 7) : piece16 ^ (tok >> 1 & (kLanes - 1)); };
    const uint32_t stages = smem_addr(sh.stage[warp]);
    auto copy = [&](int at_stage) {
        const uint32_t to = stages + at_stage * Shared::kStage;
        const int left = page < 0 ? 0 : keys - kFewGroup * ahead;
        const long long slot = page < 0 ? 0 : first_slot(a.cache, page, head) + kFewGroup * within;
        const uint8_t *k = a.cache.k_codes + (slot + tok0) * row_bytes + 16 * c;
        const uint8_t *v = a.cache.v_codes + (slot + tok0) * row_bytes + 16 * c;
        if (left >= kFewGroup && row_bytes == kRow) {  // whole: nothing to leave out, offsets known
            const uint32_t at = to + tok0 * kRow;
#pragma unroll
            for (int i = 0; i < 16; i += kEach) {
                const uint32_t to_i = at + i * kRow + 16 * swizzle(tok0 + i, c);
                cp_async16(to_i, k + i * kRow);
                cp_async16(to_i + 16 * kRow, v + i * kRow);
            }
            cp_async4(to + 32 * kRow + 4 * lane, (lane < 16 ? a.cache.k_scales : a.cache.v_scales) + (slot + (lane & 15)) * 4);
            bad &= ~(1u << at_stage);
        } else if (ahead < g1) {
            const bool in = 16 * c < row_bytes;
#pragma unroll
            for (int i = 0; i < 16; i += kEach) {
                const int tok = tok0 + i;
                const bool ok = in && tok < left;
                const uint32_t at = to + tok * kRow + 16 * swizzle(tok, c);
                cp_async16_if(at, ok ? k + i * row_bytes : a.cache.k_codes, ok);
                cp_async16_if(at + 16 * kRow, ok ? v + i * row_bytes : a.cache.v_codes, ok);
            }
            const bool ok = (lane & 15) < left;
            const uint8_t *scales = lane < 16 ? a.cache.k_scales : a.cache.v_scales;
            cp_async4_if(to + 32 * kRow + 4 * lane, ok ? scales + (slot + (lane & 15)) * 4 : scales, ok);
            bad = (bad & ~(1u << at_stage)) | (page < 0 ? 1u << at_stage : 0u);
        }
        cp_commit();
        ahead += kFewWarps, within += kFewWarps % per_page, piece += kFewWarps / per_page;
        if (within >= per_page) within -= per_page, ++piece;
        page = next_page();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy(i);

    // Query rows to fp16, each by a power of two of its own.
#pragma unroll
    for (int n = 0; n < kNR; ++n) {
        const int r = warp + kFewWarps * n;
        float v[kEachLane];
#pragma unroll
        for (int i = 0; i < kEachLane; ++i) {
            if constexpr (kNP == 2)
                v[i] = query[n][i];
            else
                v[i] = a.type == MxType::kF16 ? __half2float(__ushort_as_half(query[n][i]))
                                              : __uint_as_float((uint32_t)query[n][i] << 16);
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kEachLane; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        // 2^(141 - e) puts a largest value of biased exponent e at 2^14; not where it is infinite or NaN.
        const int e = top >= 0x7F800000u ? 141 : max((int)(top >> 23), 15);
        const float mult = __int_as_float((268 - e) << 23);
#pragma unroll
        for (int i = 0; i < kEachLane; ++i) {
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
            sees[n][j] = r < tile.rows ? min(keys_of(tile, tile.first + r, group, a.causal), keys) : 0;
        }
    }
    const float c0 = a.scale * kLog2e;
    // Keys that every row of the tile sees; rows that do not exist do not matter.
    const int all_see = min(keys_of(tile, tile.first, group, a.causal), keys);

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

    // This lane's pieces of a stage.
    uint32_t k_at[2], v_at[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) k_at[i] = (g + 8 * i) * kRow;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tok = 2 * t + (i & 1) + 8 * (i >> 1), byte = g * kVRun * kBits / 8;
        v_at[i] = (16 + tok) * kRow + 16 * swizzle(tok, byte / 16) + byte % 16;
    }
    const uint32_t mults = smem_addr(sh.mults[warp]);
    const uint32_t block_mask = blocks == 4 ? 0xFFFFFFFFu : (1u << (8 * blocks)) - 1;
    int at_stage = 0;
    for (int gi = g0 + warp; gi < g1; gi += kFewWarps) {
        cp_wait<kStages - 2>();
        __syncwarp();
        copy(at_stage == 0 ? kStages - 1 : at_stage - 1);  // into the stage used last
        const uint32_t stage = stages + at_stage * Shared::kStage;
        const int base = kFewGroup * gi, here = bad >> at_stage & 1 ? 0 : keys - base;
        at_stage = at_stage == kStages - 1 ? 0 : at_stage + 1;

        // The group's scales: the power taken out of K and V, and each token's
        // multipliers 2^(7 + exponent - power).
        uint32_t sw;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sw) : "r"(stage + 32 * kRow + 4 * lane) : "memory");
        sw &= block_mask;
        const uint32_t pair = __vmaxu2(sw & 0x00FF00FFu, sw >> 8 & 0x00FF00FFu);
        uint32_t top = max(pair & 0xFFFFu, pair >> 16);
        const bool is_v = lane >= 16;
        uint32_t any_nan = 0;  // a bit a block
        if (__any_sync(0xFFFFFFFFu, top - (134 + kVrefLow) > (uint32_t)(kVrefMax - kVrefLow))) {
            // A scale that is NaN, or one that v's powers do not reach (or that is k's).
            // NaN in v reaches the rows that see it, and no others.
            top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t e = sw >> (8 * i) & 0xFF;
                any_nan |= (e == 255) << i;
                top = max(top, e == 255 ? 0u : e);
                if (e == 255 && is_v) atomicMin(&sh.nan_from[i], base + (lane & 15));
                if (e == 255) sw &= ~(0xFFu << (8 * i));
            }
            if (__any_sync(0xFFFFFFFFu, is_v && vref_passes((int)top))) {
#pragma unroll
                for (int n = 0; n < kNR; ++n) M[n][0] = M[n][1] = kSpoiltMax, l[n][0] = l[n][1] = kSpoilt;
            }
        }
        const int ktop = (int)__reduce_max_sync(0xFFFFFFFFu, is_v ? 0u : top);
        const int vtop = (int)__reduce_max_sync(0xFFFFFFFFu, is_v ? top : 0u);
        const int kref = ktop - 134, vref = max(vtop - 134, kVrefMin);
        int ref = is_v ? vref : kref;
        const bool wide = __any_sync(0xFFFFFFFFu, top != 0 && (int)top + kWide < (is_v ? vtop : ktop));
        if (wide && top != 0) ref = is_v ? max((int)top - 134, kVrefMin) : (int)top - 134;
        {
            // fp16 exponent fields of two blocks at once: exponent - ref - 112,
            // 22 for the largest, at least 0 (then the multiplier is zero).
            const uint32_t up = (uint32_t)(512 - 112 - ref) * 0x10001u;
            uint32_t m[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                m[i] = (__vmaxu2(__byte_perm(sw, 0, i ? 0x4342 : 0x4140) + up, 0x02000200u) - 0x02000200u) << 10;
            if (any_nan) {  // zero for v; infinite for k, whose zero codes make it NaN
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((any_nan >> i & 1) && !is_v) m[i / 2] |= i % 2 ? 0x7C000000u : 0x7C00u;
            }
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(mults + 8 * lane), "r"(m[0]), "r"(m[1]) : "memory");
            __syncwarp();
        }
        uint32_t km[2], vm[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            km[i] = lds_u16(mults + 8 * (g + 8 * i) + 2 * (t * kKRun / kMxBlock)) * 0x10001u;
            const uint32_t lo = lds_u16(mults + 8 * (16 + 2 * t + 8 * i) + 2 * (g * kVRun / kMxBlock));
            const uint32_t hi = lds_u16(mults + 8 * (17 + 2 * t + 8 * i) + 2 * (g * kVRun / kMxBlock));
            vm[i] = lo | hi << 16;
        }

        // (A sum for each term: 32 sequences of 4096 in fp32 286 us, 296 with one sum.  Two sums for one term gain nothing.)
        float sc[kNP][kNR][4];
#pragma unroll
        for (int p = 0; p < kNP; ++p)
#pragma unroll
            for (int n = 0; n < kNR; ++n) sc[p][n][0] = sc[p][n][1] = sc[p][n][2] = sc[p][n][3] = 0.f;
        {
            uint32_t kw[2][kKW];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                constexpr int kPieces = kKW >= 4 ? kKW / 4 : 1;
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    const int byte = t * kKRun * kBits / 8 + 16 * j;
                    const uint32_t at = stage + k_at[i] + 16 * swizzle(g + 8 * i, byte / 16) + byte % 16;
                    if constexpr (kKW >= 4) {
                        uint32_t four[4];
                        lds_words<4>(at, four);
                        kw[i][4 * j] = four[0], kw[i][4 * j + 1] = four[1], kw[i][4 * j + 2] = four[2],
                                  kw[i][4 * j + 3] = four[3];
                    } else {
                        lds_words<kKW>(at, kw[i]);
                    }
                }
            }
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
                        mma_16816(sc[p][n], f[0][0], f[1][0], f[0][1], f[1][1], qf[p][n][k][0], qf[p][n][k][1]);
            }
            if constexpr (kNP == 2) {
#pragma unroll
                for (int n = 0; n < kNR; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[0][n][j] += sc[1][n][j];
            }
        }

        float u[kNR][4];
        bool more = false;
        float unit[2];  // 2^-vref of tokens g and g + 8
        if (!wide) {
            unit[0] = unit[1] = pow2(-vref);
#pragma unroll
            for (int n = 0; n < kNR; ++n) {
                const float f0 = c0 * pow2(power[n][0] + kref), f1 = c0 * pow2(power[n][1] + kref);
#pragma unroll
                for (int j = 0; j < 4; ++j) u[n][j] = fmaf(sc[0][n][j], j & 1 ? f1 : f0, (float)vref);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int kr = __shfl_sync(0xFFFFFFFFu, ref, g + 8 * i), vr = __shfl_sync(0xFFFFFFFFu, ref, 16 + g + 8 * i);
                unit[i] = pow2(-vr);
#pragma unroll
                for (int n = 0; n < kNR; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        u[n][2 * i + j] = fmaf(sc[0][n][2 * i + j], c0 * pow2(power[n][j] + kr), (float)vr);
            }
        }
        if (base + kFewGroup > all_see || here <= 0) {
#pragma unroll
            for (int n = 0; n < kNR; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tok = g + 8 * (j >> 1);
                    if (tok >= here || base + tok >= sees[n][j & 1]) u[n][j] = -INFINITY;
                }
        }
#pragma unroll
        for (int n = 0; n < kNR; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) more |= u[n][j] > M[n][j & 1] + kPSlack;
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
            for (int j = 0; j < 4; ++j) p[j] = ex2(u[n][j] - ((M[n][j & 1] == -INFINITY ? 0.f : M[n][j & 1]) - kPShift));
            l[n][0] = fmaf(p[0], unit[0], fmaf(p[2], unit[1], l[n][0]));
            l[n][1] = fmaf(p[1], unit[0], fmaf(p[3], unit[1], l[n][1]));
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
        uint32_t vw[4][kVW];
#pragma unroll
        for (int i = 0; i < 4; ++i) lds_words<kVW>(stage + v_at[i], vw[i]);
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
            for (int n = 0; n < kNR; ++n) {
                if constexpr (kNP == 1) {
                    mma_16816(o[n][k], f[0][0], f[0][1], f[1][0], f[1][1], pf[0][n][0], pf[0][n][1]);
                } else {
                    // A sum of the tensor cores drops what falls below its last
                    // bit: over 3750 keys a warp 6.4e-6 of the value was lost.  So
                    // each is of 16 tokens, second terms first, and added in fp32.
                    float add[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_16816(add, f[0][0], f[0][1], f[1][0], f[1][1], pf[1][n][0], pf[1][n][1]);
                    mma_16816(add, f[0][0], f[0][1], f[1][0], f[1][1], pf[0][n][0], pf[0][n][1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[n][k][j] += add[j];
                }
            }
        }
    }
    cp_wait<0>();
    __syncthreads();  // the stages have been read: their memory is the sums'

    // Sums over a warp's tokens, then over the warps, then over the cluster.
#pragma unroll
    for (int n = 0; n < kNR; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float v = l[n][j];
#pragma unroll
            for (int x = 4; x < 32; x *= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, x);
            const int r = 8 * n + 2 * t + j;
            // A code of v that is NaN reaches rows that do not see it here: they have NaN among their values, but not in their sum.
            float any = 0.f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) any += o[n][i][j] + o[n][i][2 + j];
            if (__ballot_sync(0xFFFFFFFFu, isnan(any) && !isnan(v)) >> t & 0x11111111u) M[n][j] = kSpoiltMax, v = kSpoilt;
            if (g == 0) sh.m[warp][r] = M[n][j], sh.l[warp][r] = v;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                *reinterpret_cast<float2 *>(&sh.o[warp][r][g * kVRun + 2 * (i ^ sum_swizzle<kDP>(r, g))]) =
                    make_float2(o[n][i][j], o[n][i][2 + j]);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < tile.rows * (kDP / 4); i += kThreads) {
        const int r = i / (kDP / 4), d = 4 * (i % (kDP / 4));
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, sh.m[w][r]);
        Joined sum;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w)
            sum.add(sh.m[w][r], m, sh.l[w][r], *reinterpret_cast<const float4 *>(&sh.o[w][r][sum_place<kDP>(r, d)]));
        if (sum_swizzle<kDP>(r, d / kVRun) & 1) sum.o = make_float4(sum.o.z, sum.o.w, sum.o.x, sum.o.y);
        *reinterpret_cast<float4 *>(&sh.o[0][r][sum_place<kDP>(r, d)]) = sum.o;
        if (d == 0) sh.m_all[r] = m, sh.l_all[r] = sum.l;
    }
    if (S > 1)
        cluster_sync_all();
    else
        __syncthreads();
    const uint32_t o_at = smem_addr(sh.o), m_at = smem_addr(sh.m_all), l_at = smem_addr(sh.l_all),
                   n_at = smem_addr(sh.nan_from);
    float *ws = parts > 1 ? a.workspace + (size_t)(blockIdx.x / S) * few_part_floats(kR, kDP) : nullptr;
    bool spoilt = false;
    for (int i = rank * kThreads + threadIdx.x; i < tile.rows * (kDP / 4); i += S * kThreads) {
        const int r = i / (kDP / 4), d = 4 * (i % (kDP / 4));
        if (d >= D) continue;
        float m = -INFINITY;
        int nan_from = kNever;
        for (int s = 0; s < S; ++s) {
            m = fmaxf(m, ld_cluster_f32(map_to_rank(m_at + 4 * r, s)));
            nan_from = min(nan_from, __float_as_int(ld_cluster_f32(map_to_rank(n_at + 4 * (d / kMxBlock), s))));
        }
        Joined sum;
        for (int s = 0; s < S; ++s)
            sum.add(ld_cluster_f32(map_to_rank(m_at + 4 * r, s)), m, ld_cluster_f32(map_to_rank(l_at + 4 * r, s)),
                    ld_cluster_v4(map_to_rank(o_at + 4 * (r * kDP + sum_place<kDP>(r, d)), s)));
        if (parts > 1) {
            *reinterpret_cast<float4 *>(ws + r * kDP + d) = sum.o;
            if (d == 0) ws[kR * kDP + r] = m, ws[kR * (kDP + 1) + r] = sum.l;
            if (r == 0 && d % kMxBlock == 0) ws[kR * (kDP + 2) + d / kMxBlock] = __int_as_float(nan_from);
        } else {
            const int row = tile.first + r;
            sum.store(a, tile, row, head, group, d, nan_from);
            spoilt |= sum.l == kSpoilt;
        }
    }
    if (S > 1) cluster_sync_all();  // no CTA leaves while another reads its sums
    if (__syncthreads_or(spoilt))
        few_plain<kBits, kR, kThreads / (kDP / 4)>(a, group, blockIdx.x / cluster_size(), (int)cluster_rank(),
                                                   (int)cluster_size(), *reinterpret_cast<PlainScratch *>(raw));
}

// Joins the parts of a tile's keys that the clusters left in the workspace.
template <int kBits, int kDP, int kNR>
__global__ void __launch_bounds__(kJoinThreads) mx_attention_join_kernel(const __grid_constant__ MxAttentionArgs a,
                                                                         const int group, const int parts) {
    __shared__ __align__(16) PlainScratch scratch;
    bool spoilt = false;
    constexpr int kR = 8 * kNR;
    pdl_wait();
    const int head = (int)(blockIdx.x % a.cache.heads);
    const RowTile tile = row_tile(a.batch, blockIdx.x / a.cache.heads, group, kR, a.tokens);
    const float *ws = a.workspace + (size_t)blockIdx.x * parts * few_part_floats(kR, kDP);
    for (int i = threadIdx.x; i < tile.rows * (kDP / 4); i += kJoinThreads) {
        const int r = i / (kDP / 4), d = 4 * (i % (kDP / 4));
        if (d >= a.cache.D) continue;
        float m = -INFINITY;
        int nan_from = kNever;
#pragma unroll 8
        for (int s = 0; s < parts; ++s) {
            const float *w = ws + s * few_part_floats(kR, kDP);
            m = fmaxf(m, w[kR * kDP + r]);
            nan_from = min(nan_from, __float_as_int(w[kR * (kDP + 2) + d / kMxBlock]));
        }
        Joined sum;
#pragma unroll 8
        for (int s = 0; s < parts; ++s) {
            const float *w = ws + s * few_part_floats(kR, kDP);
            sum.add(w[kR * kDP + r], m, w[kR * (kDP + 1) + r], *reinterpret_cast<const float4 *>(w + r * kDP + d));
        }
        const int row = tile.first + r;
        sum.store(a, tile, row, head, group, d, nan_from);
        spoilt |= sum.l == kSpoilt;
    }
    if (__syncthreads_or(spoilt)) few_plain<kBits, kR, kR>(a, group, blockIdx.x, 0, 1, scratch);
}

template <int kBits, int kDP, int kNR, int kNP>
cudaError_t launch_few(const LaunchCtx &c, const MxAttentionArgs &a, const FewSplit &f) {
    auto kernel = mx_attention_few_kernel<kBits, kDP, kNR, kNP>;
    constexpr size_t bytes = sizeof(FewShared<kBits, kDP, kNR, kNP>);
    cudaError_t e = ensure_smem(kernel, bytes);
    if (e != cudaSuccess) return e;
    const int group = a.heads / a.cache.heads;
    const long long tiles = few_tiles(a.tokens, group, kNR, a.batch.seqs);
    const long long ctas = tiles * a.cache.heads * f.parts * f.cluster;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = f.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.pdl ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, group, f.parts);
    if (e != cudaSuccess || f.parts == 1) return e;
    return launch_kernel(c, mx_attention_join_kernel<kBits, kDP, kNR>, dim3((unsigned)(tiles * a.cache.heads)), dim3(kJoinThreads),
                         0, a, group, f.parts);
}

template <int kBits, int kDP>
cudaError_t launch_rows(const LaunchCtx &c, const MxAttentionArgs &a, const FewSplit &f, bool as_f32) {
    if (as_f32 || a.type == MxType::kF32) return f.rows_8 == 2 ? launch_few<kBits, kDP, 2, 2>(c, a, f) : launch_few<kBits, kDP, 1, 2>(c, a, f);
    return f.rows_8 == 2 ? launch_few<kBits, kDP, 2, 1>(c, a, f) : launch_few<kBits, kDP, 1, 1>(c, a, f);
}

}  // namespace

size_t mx_attention_few_workspace(int tokens, int heads, int kv_heads, int D, int seqs, const FewSplit &f) {
    if (f.parts == 1) return 0;
    const size_t tiles = few_tiles(tokens, heads / kv_heads, f.rows_8, seqs);
    return tiles * kv_heads * f.parts * few_part_floats(8 * f.rows_8, D <= 64 ? 64 : 128) * sizeof(float);
}

cudaError_t launch_mx_attention_few(const LaunchCtx &c, const MxAttentionArgs &a, const FewSplit &f, bool as_f32) {
    const bool narrow = a.cache.D <= 64;
    if (a.cache.bits == 4) return narrow ? launch_rows<4, 64>(c, a, f, as_f32) : launch_rows<4, 128>(c, a, f, as_f32);
    return narrow ? launch_rows<8, 64>(c, a, f, as_f32) : launch_rows<8, 128>(c, a, f, as_f32);
}

}  // namespace q4mm

// y[t][n] = sum_k x[t][k]·w[n][k] of microscaled operands on the tensor cores
// (tcgen05 block-scaled MMA, sm_103a): w in E2M1, x in E2M1 (kX8 = false,
// kind::mxf4, K = 64 per instruction) or E4M3 (kX8 = true, kind::mxf8f6f4,
// K = 32).  The hardware multiplies the codes, applies both blocks' scales
// and adds in fp32; nothing is dequantised in registers.
//
// The weights are the MMA's A operand (M = 128 rows), the tokens its B
// operand (N = kTok tokens), so a call with few tokens wastes no tensor rows:
// D[row][token] lies in tensor memory with a weight row per lane, and a
// warp's 32 lanes hold 32 consecutive n of one token, a contiguous run of y.
//
// A stage of the ring holds 128 bytes of shared memory per row: 256 values of
// K of packed E2M1, or 128 values with kX8, where the 4-bit weights are
// unpacked by the tensor copy itself into the 16-bytes-per-16-values form
// that the mixed MMA reads.  Either way it is four MMAs.  Block scales come
// as whole 512-byte tiles by plain bulk copies and go on to tensor memory,
// where the MMA takes them from a multiple of four columns on.
//
// Two forms, chosen by mx_geometry.h from estimates of both:
//  * mx_mm_split_kernel, up to 128 tokens a tile, K split over a cluster.  A
//    call with few tokens reads its weights once and is bound by them and by
//    the chain of latencies around them: 4096 x 4096 at one token takes 4.2
//    us (x in 4 bits) and 4.8 (8 bits, whose unpacking copies move 64 bytes
//    a row) in a chain of calls, of which 1.3 us are the weights' at the
//    copy rate, 2.9 a small product's (1024 x 1024; 128 x 128 unsplit 1.9).
//    Tiles are dealt whole, so a width whose tiles do not fill whole rounds
//    of SMs is bound by the SMs that take one more: 4096 -> 22016, 172 tiles
//    on 152 SMs, 10.2 and 12.2 us where the bytes take 7.1, against 16384 ->
//    38912, two tiles to every SM, 52 and 55 us, 6.5 and 6.2 TB/s.
//  * mx_mm_pair_kernel, 256 rows x 256 tokens on a pair of CTAs, for the
//    rest.  8192 tokens 4096 -> 11008: 112 us in 4 bits (6.6 PFLOP/s), 206 in
//    8 (3.6); 8192 tokens 8192 -> 8192: 147 us (7.5 PFLOP/s).  Bound by the
//    tensor pipe (four MMAs of 256 tokens of a 4-bit stage alone run 620
//    cycles where 512 are nominal), by some 900 cycles between two tiles and
//    by the last, partly filled round of tiles; kept busy for seconds, by
//    the board's power limit.  Small tiles of tokens are bound by the fixed
//    work of a stage and the launch, and, where there are fewer tiles than
//    pairs, by the stages that each walks one after the other, since pairs
//    do not split K (300 tokens 11008 -> 4096 in 8 bits: 64 tiles, 19.7 us).
//
// Tensor memory: every CTA of a grid has its columns before it lets the next
// grid on the stream start, and grids of this library on different streams
// share an SM only where the columns of both fit, which their shared memory
// sees to (kernels.h): a CTA of the split form takes at most 256 columns and
// some 100 KB, one of a pair all columns and all shared memory.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>
#include <mutex>

#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "mx_geometry.h"
#include "sync.cuh"

namespace q4mm {

namespace {

constexpr int kMmRows = 128;                 // weight rows per CTA: the MMA's M
constexpr int kMmThreads = 192;              // producer, MMA issuer, 4 epilogue warps
constexpr uint32_t kMmWBytes = kMmRows * 128;  // weight operand bytes per stage

template <bool kX8, int kTok>
struct MmLayout {
    static constexpr int kStageK = kX8 ? 128 : 256;
    static constexpr int kScaleTiles = kStageK / 128;                 // scale tiles per 128 rows and stage
    // Bytes that the weight copy reports to its barrier: the unpacking copy
    // counts what it reads, half of what it lays out.
    static constexpr uint32_t w_tx = kX8 ? kMmWBytes / 2 : kMmWBytes;
    static constexpr uint32_t off_x = kMmWBytes;
    static constexpr uint32_t off_sw = off_x + kTok * 128;
    static constexpr uint32_t off_sx = off_sw + kScaleTiles * kMxTileBytes;
    static constexpr uint32_t stage = (off_sx + kScaleTiles * kMxTileBytes + 1023) / 1024 * 1024;
    // Two CTAs per SM: half of the 227 KB each.
    static constexpr int kStages = (int)(112 * 1024 / stage);
    static constexpr uint32_t off_bar = kStages * stage;
    static constexpr uint32_t total = off_bar + 8 * (2 * kStages + 1) + 16 + 1024;
    // Tensor memory columns: the accumulator, then the scales of a stage.
    static constexpr int kColSw = kTok < 32 ? 32 : kTok;
    static constexpr int kColSx = kColSw + 4 * kScaleTiles;
    static constexpr int kColsUsed = kColSx + 4 * kScaleTiles;
    static constexpr int kCols = kColsUsed <= 64 ? 64 : kColsUsed <= 128 ? 128 : 256;
    static_assert(kStages >= 2 && kStages <= 8 && 2 * (total + 1024) <= 233472, "two CTAs per SM");
    static_assert(2 * kCols <= 512 && total + kCtaSharedExtra >= kHalfTmemShared, "tensor memory of two CTAs");
    static_assert(kTok <= kMxTileRows && kTok * kMmRows * 4 <= off_bar, "partial sums fit the ring");
};

// Shared-memory matrix descriptors: K-major rows of 128 bytes in 8-row atoms
// with the 128-byte swizzle, and the 32 x 16-byte scale tile (8-row groups of
// 128 bytes, no swizzle).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(128u >> 4) << 32 | (uint64_t)1u << 46;
}

// Block-scaled instruction descriptor: E8M0 scales, K-major operands, M = m.
// sf: which byte of a scale column's 32-bit word the instruction starts at.
template <bool kX8>
__device__ __forceinline__ uint32_t mx_idesc(int n, int sf, int m = kMmRows) {
    const uint32_t a_fmt = kX8 ? 5u : 1u;  // E2M1
    const uint32_t b_fmt = kX8 ? 0u : 1u;  // E4M3 or E2M1
    return (uint32_t)sf << 4 | a_fmt << 7 | b_fmt << 10 | (uint32_t)(n >> 3) << 17 | 1u << 23 |
           (uint32_t)(m >> 4) << 24 | (uint32_t)sf << 29;
}

template <bool kX8, int kGroup>
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t accumulate) {
#define Q4MM_MX_MMA(group, kind, vec)                                                                             \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                  \
                 "tcgen05.mma.cta_group::" group ".kind::" kind ".block_scale.scale_vec::" vec                       \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                                \
                 "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                                      \
                 : "memory")
    if constexpr (kX8 && kGroup == 1) Q4MM_MX_MMA("1", "mxf8f6f4", "1X");
    if constexpr (!kX8 && kGroup == 1) Q4MM_MX_MMA("1", "mxf4", "2X");
    if constexpr (kX8 && kGroup == 2) Q4MM_MX_MMA("2", "mxf8f6f4", "1X");
    if constexpr (!kX8 && kGroup == 2) Q4MM_MX_MMA("2", "mxf4", "2X");
#undef Q4MM_MX_MMA
}

// A 128-row scale tile to four tensor-memory columns, repeated in the four
// lane quarters.
__device__ __forceinline__ void scale_to_tmem(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void mm_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void mm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void mm_tma_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_addr(bar))
        : "memory");
}

// Eight columns of this thread's tensor-memory lane.
__device__ __forceinline__ void mm_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// True in one lane of the converged warp, the same one each time.
__device__ __forceinline__ bool elect_lane() {
    uint32_t mine;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(mine));
    return mine != 0;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Up to four consecutive n of one token; one store where all four are there
// and aligned.
template <class T>
__device__ __forceinline__ void store_y4(T *p, int left, float4 v) {
    const float e[4] = {v.x, v.y, v.z, v.w};
    if (left >= 4 && reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4 *>(p) = v;
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(mx_pack2<T>(v.x, v.y), mx_pack2<T>(v.z, v.w));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = mx_from_float<T>(e[i]);
    }
}

__device__ __forceinline__ void store_y(void *y, MxType type, size_t at, float v) {
    if (type == MxType::kF32)
        static_cast<float *>(y)[at] = v;
    else if (type == MxType::kF16)
        static_cast<__half *>(y)[at] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(y)[at] = __float2bfloat16_rn(v);
}

// Up to 128 tokens per tile, K split over the CTAs of a cluster: rank r of S
// takes the stages [r·c/S, (r+1)·c/S) and puts its partial sums, [token][row],
// into its shared memory, over the ring; rank s then adds the S partial sums
// of rows 4·floor(32·s/S) onwards in rank order, read over the cluster eight
// loads at a time, and writes y, so the result does not depend on scheduling.
// (Pushed to their owner with st.async instead, the sums of 16 tokens of a
// 4096 x 4096 product take 0.6 us longer, those of 128 tokens 11.)
template <bool kX8, int kTok>
__global__ void __launch_bounds__(kMmThreads, 2)
    mx_mm_split_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const uint8_t *__restrict__ w_scales, const uint8_t *__restrict__ x_scales,
                       void *__restrict__ y, MxType type, int K, int N, int T, int n_mma, int *status,
                       long long wait_limit, int withhold) {
    using L = MmLayout<kX8, kTok>;
    extern __shared__ uint8_t mm_smem_raw[];
    __shared__ volatile int abort_flag;
    const uint32_t raw = smem_addr(mm_smem_raw);
    uint8_t *smem = mm_smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_addr(smem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::off_bar), *empty = full + L::kStages;
    uint64_t *done = empty + L::kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int Kp = mx_padded(K), nkt = Kp / kMxPadK;
    const int row_tile = blockIdx.x / S, row0 = row_tile * kMmRows, tok0 = blockIdx.y * kTok;
    const int all = (Kp + L::kStageK - 1) / L::kStageK;
    const int c_lo = (int)((long long)rank * all / S), chunks = (int)((long long)(rank + 1) * all / S) - c_lo;
    const int toks = min(kTok, T - tok0);

    // Four copies per stage, one per lane: a bulk copy holds the thread that
    // issues it for some 475 cycles (measured), but lanes that issue by one
    // instruction do so side by side.  Copy j of a stage: weights and tokens
    // (tensor copies), their scales (plain ones).
    auto issue = [&](int c, int j, bool here) {
        const int s = c % L::kStages;
        const int k0 = (c_lo + c) * L::kStageK, kt = (c_lo + c) * L::kScaleTiles;
        const uint32_t sbytes = (uint32_t)min(L::kScaleTiles, nkt - kt) * kMxTileBytes;
        here = here && c != withhold;  // (test only: a stage that never arrives)
        if (here && j == 0) mbar_arrive_expect_tx(&full[s], L::w_tx + n_mma * 128 + 2 * sbytes);
        __syncwarp();
        const int c0 = kX8 ? k0 : k0 / 2;  // 8-bit codes and unpacked 4-bit ones in values, else bytes
        if (here && j < 2)
            mm_tma_2d(sbase + s * L::stage + (j ? L::off_x : 0u), j ? &tm_x : &tm_w, c0, j ? tok0 : row0, &full[s]);
        if (here && j >= 2)
            bulk_g2s(smem + s * L::stage + (j == 3 ? L::off_sx : L::off_sw),
                     (j == 3 ? x_scales + (size_t)(tok0 / kMxTileRows) * nkt * kMxTileBytes
                             : w_scales + (size_t)row_tile * nkt * kMxTileBytes) + (size_t)kt * kMxTileBytes,
                     sbytes, &full[s]);
        __syncwarp();
    };
    const int lap = min(chunks, L::kStages);

    if (warp == 0) {
        if (lane == 0) {
            for (int s = 0; s < L::kStages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            mbar_init(done, 1);
            abort_flag = 0;
            fence_mbar_init();
            prefetch_map(&tm_w);
            prefetch_map(&tm_x);
        }
        __syncwarp();
        // Every operand may come from the previous kernel on the stream, the
        // weights too (a quantisation is a kernel like any other): copies
        // start after it.
        pdl_wait();
        issue(lane >> 2, lane & 3, (lane >> 2) < lap);
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(L::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    mm_fence_before();
    __syncthreads();
    mm_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();

    if (warp == 0) {
        int c = lap;
        for (; c < chunks; ++c) {
            const bool ok =
                mbar_wait_abortable(&empty[c % L::kStages], ((c / L::kStages) - 1) & 1, wait_limit, &abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) {
                    abort_flag = 1;
                    flag_timeout(status);
                }
                break;
            }
            issue(c, lane, lane < 4);
        }
        // No copy may still be writing shared memory at exit.
        if (lane == 0)
            for (int i = max(0, c - L::kStages); i < c; ++i)
                if (i != withhold) (void)mbar_wait_bounded(&full[i % L::kStages], (i / L::kStages) & 1, wait_limit);
        __syncwarp();
    } else if (warp == 1) {
        // The whole warp takes the loop and one lane issues, so that addresses
        // and descriptors stay in uniform registers, where the MMAs want them.
        const bool leader = elect_lane();
        for (int c = 0; c < chunks; ++c) {
            const int s = c % L::kStages;
            if (!__all_sync(0xffffffffu,
                            mbar_spin_abortable(&full[s], (c / L::kStages) & 1, wait_limit, &abort_flag))) {
                if (leader) {
                    abort_flag = 1;
                    flag_timeout(status);
                }
                break;
            }
            mm_fence_after();
            const uint32_t sa = sbase + s * L::stage;
            const int kts = min(L::kScaleTiles, nkt - (c_lo + c) * L::kScaleTiles);
            const uint64_t ad = sw128_desc(sa), bd = sw128_desc(sa + L::off_x);
            if (leader) {
#pragma unroll
                for (int j = 0; j < L::kScaleTiles; ++j) {
                    if (j >= kts) break;
                    scale_to_tmem(tmem + L::kColSw + 4 * j, scale_desc(sa + L::off_sw + j * kMxTileBytes));
                    scale_to_tmem(tmem + L::kColSx + 4 * j, scale_desc(sa + L::off_sx + j * kMxTileBytes));
                }
                // 32 bytes of each row per MMA: with kX8 32 values and one scale
                // byte, else 64 values and two.
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int j = kX8 ? 0 : m / 2, sf = kX8 ? m : 2 * (m % 2);
                    if (j < kts)
                        mx_mma<kX8, 1>(tmem, ad + 2 * m, bd + 2 * m, mx_idesc<kX8>(n_mma, sf), tmem + L::kColSw + 4 * j,
                                       tmem + L::kColSx + 4 * j, (c | m) != 0);
                }
                mm_commit(&empty[s]);
            }
            __syncwarp();
        }
        // Whatever was issued completes before tensor memory is read or freed.
        if (leader) mm_commit(done);
        __syncwarp();
        (void)mbar_wait_bounded(done, 0, wait_limit);
        __syncwarp();
    }
    // (The producer and the issuer leave their branches through a reconverged
    // warp; every warp takes part from here on.)
    const bool ok = __syncthreads_and(mbar_wait_bounded(done, 0, wait_limit) ? 1 : 0) != 0 && !abort_flag;
    mm_fence_after();
    pdl_wait();  // y may still be read by the previous kernel
    float *part = reinterpret_cast<float *>(smem);  // [token][128 rows]
    if (warp >= 2) {
        const int q = warp & 3;  // tensor-memory lane quarter of this warp
        const int r = 32 * q + lane, n = row0 + r;
        for (int t = 0; t < toks; t += 8) {
            float v[8];
            if (ok && chunks > 0) {
                mm_ld8(tmem + ((uint32_t)(32 * q) << 16) + t, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.f;
            }
            if (S > 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (t + i < toks) part[(t + i) * kMmRows + r] = v[i];
            } else if (ok && n < N) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (t + i < toks) store_y(y, type, (size_t)(tok0 + t + i) * N + n, v[i]);
            }
            __syncwarp();
        }
        mm_fence_before();
    }
    if (S > 1) {
        cluster_arrive();
        cluster_wait();
        const int lo = mx_first_row(rank, S), rows4 = (mx_first_row(rank + 1, S) - lo) / 4;
        for (int i = threadIdx.x; i < rows4 * toks; i += kMmThreads) {
            const int r = lo + 4 * (i % rows4), t = i / rows4;
            const uint32_t at = smem_addr(part + t * kMmRows + r);
            float4 v[kMxMaxSplit];
#pragma unroll
            for (int s = 0; s < kMxMaxSplit; ++s)
                if (s < S) v[s] = ld_cluster_v4(map_to_rank(at, (uint32_t)s));
            float4 acc = v[0];
#pragma unroll
            for (int s = 1; s < kMxMaxSplit; ++s)
                if (s < S) acc.x += v[s].x, acc.y += v[s].y, acc.z += v[s].z, acc.w += v[s].w;
            const size_t to = (size_t)(tok0 + t) * N + row0 + r;
            if (type == MxType::kF32)
                store_y4(static_cast<float *>(y) + to, N - row0 - r, acc);
            else if (type == MxType::kF16)
                store_y4(static_cast<__half *>(y) + to, N - row0 - r, acc);
            else
                store_y4(static_cast<__nv_bfloat16 *>(y) + to, N - row0 - r, acc);
        }
        __syncwarp();
        cluster_arrive();  // this CTA has read its peers' sums
    }
    __syncthreads();
    if (warp == 1) {
        mm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
    }
    if (S > 1) cluster_wait();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------------------
// Many tokens: CTA pairs (cta_group::2), 256 weight rows x up to 256 tokens.
// ---------------------------------------------------------------------------

// Warps: operand copies, MMA issuer, 2 x 4 for the scales, the epilogue's (three
// for each lane quarter: with 256 tokens the accumulators share three blocks
// of 32 columns), scale copies.
constexpr int kPairEpiWarp = 10, kPairEpi = 3, kPairCopyWarp = kPairEpiWarp + 4 * kPairEpi;
constexpr int kPairThreads = 32 * (kPairCopyWarp + 1);

// kSub: blocks of 128 bytes of K per row and stage.  A stage costs its warps
// some 400 cycles each besides the MMAs, more than four MMAs of a small tile
// last: tiles of up to 128 tokens take two blocks a stage.
template <bool kX8, int kSub>
struct PairLayout {
    static constexpr int kTok = kSub == 1 ? 256 : kMxPairTwoBlocks;
    static constexpr int kStages = kSub == 1 ? 6 : 4;
    static constexpr int kXTiles = kSub == 1 ? 3 : 2;  // 128-row scale tiles that a tile's tokens touch at most
    static constexpr int kStageK = kSub * (kX8 ? 128 : 256);
    static constexpr int kScaleTiles = kStageK / 128;
    static constexpr uint32_t w_tx = kX8 ? kMmWBytes / 2 : kMmWBytes;  // of a block
    static constexpr uint32_t x_block = kTok / 2 * 128;
    static constexpr uint32_t off_x = kSub * kMmWBytes;
    static constexpr uint32_t off_sw = off_x + kSub * x_block;
    static constexpr uint32_t off_sx = off_sw + kScaleTiles * kMxTileBytes;
    static constexpr uint32_t stage = (off_sx + kXTiles * kScaleTiles * kMxTileBytes + 1023) / 1024 * 1024;
    // Tensor memory: accumulators of up to kTok columns at 0 and at kCol1,
    // which share what reaches past kCol1, then the scale buffers: per 128
    // values of K four columns for w and one for 32 tokens.
    static constexpr int kCol1 = kSub == 1 ? 160 : 128;
    static constexpr int kColScales = kCol1 + kTok;
    static constexpr int kXCols = kTok / 32;
    static constexpr int kScaleCols = kScaleTiles * (4 + kXCols);
    static constexpr int kScaleRoom = (512 - kColScales) / kScaleCols;
    static constexpr int kScaleBufs = kScaleRoom < kStages ? kScaleRoom : kStages;
    static constexpr uint32_t off_bar = kStages * stage;
    static constexpr int kBars = 3 * kStages + 5;
    static constexpr uint32_t total = off_bar + 8 * kBars + 16 + 1024;
    static_assert(total <= 232448, "shared memory");
    static_assert(total + kCtaSharedExtra + kHalfTmemShared > kSmShared, "tensor memory for itself");
    static_assert(kScaleBufs >= 3, "scale buffers");
};

__device__ __forceinline__ void pair_tma_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Arrives on the barrier at this offset in both CTAs of the pair once the
// MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// Arrives on a barrier of either CTA of the pair, at cluster scope.  What the
// arrival hands over lies in tensor memory alone (scales written, accumulators
// read): those accesses are complete before it (tcgen05.wait) and ordered by
// the tcgen05 fences on both sides, so it orders no other memory and is
// relaxed (the scale tiles read in shared memory are what was written).
// (Releasing at cluster scope it took about a microsecond: 326 us
// for 8192 tokens 4096 -> 11008 instead of the 162 of that build.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Test of a phase that arrivals and copies of both CTAs complete: at cluster
// scope.
__device__ __forceinline__ bool pair_test_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool pair_spin(uint64_t *bar, uint32_t parity, long long limit_cycles,
                                          const volatile int *abort) {
    if (pair_test_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
        if (pair_test_wait(bar, parity)) return true;
        if (*abort || clock64() - t0 > limit_cycles) return false;
    }
}

__device__ __forceinline__ void mm_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// One n of `count` consecutive tokens, N values apart.  The stores are
// unrolled; two copies of the loop in the kernel cost a tile a microsecond
// (instruction cache), and one loop for all types, with an index for every
// store, more than that.
template <class T>
__device__ __forceinline__ void store_column(T *p, int N, int count, const float (&v)[32]) {
    if (count >= 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) p[(size_t)i * N] = mx_from_float<T>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < count) p[(size_t)i * N] = mx_from_float<T>(v[i]);
    }
}

// The tile of a running index: token tiles in groups of 8, row tiles outside
// the group's tokens, so that the tiles in flight share operands in L2.
struct PairTile {
    int row0, tok0;
};
__device__ __forceinline__ PairTile pair_tile(long long i, int row_tiles, int tok_tiles, int tile_tok) {
    const long long per_group = 8LL * row_tiles;
    const int g = (int)(i / per_group), in = (int)(i % per_group);
    const int width = min(8, tok_tiles - 8 * g);
    return PairTile{in / width * 2 * kMmRows, (8 * g + in % width) * tile_tok};
}

// 4, 8 or 16 columns of this thread's tensor-memory lane.
template <int kN>
__device__ __forceinline__ void mm_st(uint32_t taddr, const uint32_t (&r)[kN]) {
    static_assert(kN == 4 || kN == 8 || kN == 16, "columns");
    if constexpr (kN == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3])
                     : "memory");
    if constexpr (kN == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    if constexpr (kN == 16)
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15, %16};" ::"r"(taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
            "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
            : "memory");
}

// A cluster of two CTAs computes 256 weight rows x tile_tok tokens with
// instructions of M = 256: each CTA stages its 128 weight rows and its half
// of the tokens, and holds its 128 rows of D.  Half of the operand bytes of
// two single CTAs, both from L2 and in shared memory.  The pair takes every
// (number of pairs)-th tile; the epilogue of a tile runs beside the MMAs of
// the next, whose accumulator shares three blocks of 32 columns with it (the
// scales need the rest).  All operand copies of both CTAs are counted on the
// leader's barriers, and its one thread issues every MMA; completions are
// multicast to both.  What was measured on the way (8192 tokens 4096 -> 11008
// in 4 bits): scales by tcgen05.cp 230 us, by scale warps whose arrival
// releases at cluster scope 326, by the plain arrival 162, copies issued by
// lanes 142, one barrier a stage 130, shared columns read first 118, the
// issuing warp converged 111.
template <bool kX8, int kSub>
__global__ void __launch_bounds__(kPairThreads, 1)
    mx_mm_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const uint8_t *__restrict__ w_scales, const uint8_t *__restrict__ x_scales,
                      void *__restrict__ y, MxType type, int K, int N, int T, int tile_tok, int x_tiles, int row_tiles,
                      int tok_tiles, int *status, long long wait_limit, int withhold) {
    using L = PairLayout<kX8, kSub>;
    extern __shared__ uint8_t mm_smem_raw[];
    __shared__ volatile int abort_flag;
    const uint32_t raw = smem_addr(mm_smem_raw);
    uint8_t *smem = mm_smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_addr(smem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::off_bar), *empty = full + L::kStages;
    uint64_t *scales_in = empty + L::kStages;  // a stage's scale tiles have landed in this CTA's shared memory
    uint64_t *acc_full = scales_in + L::kStages, *acc_free = acc_full + 2;  // one of each per accumulator
    uint64_t *done = acc_free + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int Kp = mx_padded(K), nkt = Kp / kMxPadK;
    const int chunks = (Kp + L::kStageK - 1) / L::kStageK;
    const long long tiles = (long long)row_tiles * tok_tiles;
    const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    // Blocks of 32 tokens that the two accumulators share.
    const int blocks = tile_tok / 32, shared = max(0, blocks - L::kCol1 / 32);

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1 + 8);  // both CTAs' operands (bytes), 4 scale warps of each
            mbar_init(&empty[s], 1);
            mbar_init(&scales_in[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_free[b], 2 * 4 * kPairEpi);  // of both CTAs
        }
        mbar_init(done, 1);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_map(&tm_w);
        prefetch_map(&tm_x);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    mm_fence_before();
    __syncthreads();
    cluster_sync_all();
    mm_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    if (warp == 0 || warp == kPairCopyWarp) {
        // Two warps copy a stage in, one copy per lane and the lanes by
        // one instruction (a copy holds the thread that issues it for some
        // 475 cycles): the first the weights and the tokens, the other the
        // scales of the weights (lane 0) and of the tokens (up to three).
        const bool operands = warp == 0;
        int s = 0;
        uint32_t ph = 1;  // a fresh barrier's previous phase counts as done
        long long n = 0;  // stages issued
        bool ok = true;
        const uint32_t tx = 2 * (L::w_tx + (uint32_t)tile_tok / 2 * 128);  // a block of both CTAs
        const int blocks_k = (Kp + L::kStageK / kSub - 1) / (L::kStageK / kSub);
        const int w_all = (N + kMxTileRows - 1) / kMxTileRows, x_all = (T + kMxTileRows - 1) / kMxTileRows;
        for (long long i = pair; i < tiles && ok; i += pairs) {
            const PairTile t = pair_tile(i, row_tiles, tok_tiles, tile_tok);
            const int wrow = t.row0 + rank * kMmRows, xrow = t.tok0 + rank * (tile_tok / 2);
            // Lanes 0 to kSub - 1: blocks of the weights, then of the tokens.
            const bool of_x = lane >= kSub;
            const int sub = of_x ? lane - kSub : lane;
            const CUtensorMap *map = of_x ? &tm_x : &tm_w;
            const int crow = of_x ? xrow : wrow;
            const uint32_t to = of_x ? L::off_x + sub * L::x_block : sub * kMmWBytes;
            // Scale tiles: this CTA's rows (none past the last row) and all
            // of the tile's tokens.
            const int wt = wrow / kMxTileRows, nw = wt < w_all ? 1 : 0;
            const int xt = t.tok0 / kMxTileRows, nx = min(x_tiles, x_all - xt);
            const uint8_t *from = lane == 0 ? w_scales + (size_t)wt * nkt * kMxTileBytes
                                            : x_scales + (size_t)(xt + lane - 1) * nkt * kMxTileBytes;
            const bool mine = operands ? lane < 2 * kSub : lane == 0 ? nw != 0 : lane <= nx;
            for (int c = 0; c < chunks; ++c, ++n) {
                ok = mbar_wait_abortable(&empty[s], ph, wait_limit, &abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) {
                        abort_flag = 1;
                        flag_timeout(status);
                    }
                    ok = false;
                    break;
                }
                const bool here = n != withhold;  // (test only: a stage that never arrives)
                const uint32_t off = s * L::stage;
                if (operands) {
                    const uint32_t bar = map_to_rank(smem_addr(&full[s]), 0);  // the leader's
                    const int here_k = min(kSub, blocks_k - c * kSub);
                    if (here && lane == 0 && rank == 0) mbar_arrive_expect_tx(&full[s], here_k * tx);
                    // (128 values or, packed, 128 bytes.)
                    if (here && mine && sub < here_k)
                        pair_tma_2d(sbase + off + to, map, (c * kSub + sub) * 128, crow, bar);
                } else {
                    const int kt = c * L::kScaleTiles;
                    const uint32_t sbytes = (uint32_t)min(L::kScaleTiles, nkt - kt) * kMxTileBytes;
                    if (here && lane == 0) mbar_arrive_expect_tx(&scales_in[s], (uint32_t)(nw + nx) * sbytes);
                    __syncwarp();
                    if (here && mine)
                        bulk_g2s(smem + off + (lane ? L::off_sx + (lane - 1) * L::kScaleTiles * kMxTileBytes : L::off_sw),
                                 from + (size_t)kt * kMxTileBytes, sbytes, &scales_in[s]);
                }
                __syncwarp();
                if (++s == L::kStages) s = 0, ph ^= 1u;
            }
        }
        // No copy may still be writing shared memory at exit: the MMAs wait
        // for every stage, and their completion is awaited here.  After a
        // time-out, which leaves copies that nobody waits for (they count on
        // the other CTA's barriers), give them far longer than a copy takes.
        for (int k = 0; k < L::kStages && ok; ++k) {
            ok = __all_sync(0xffffffffu, mbar_wait_abortable(&empty[s], ph, wait_limit, &abort_flag) ? 1 : 0) != 0;
            if (++s == L::kStages) s = 0, ph ^= 1u;
        }
        if (!ok) {
            if (lane == 0) abort_flag = 1;
            outlast_copies();
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // What this warp does between MMAs is time that the tensor pipe
            // may run dry (it queues little more than one MMA): one barrier
            // per stage, tested as soon as the stage before is issued.  The
            // whole warp takes the loop and one lane issues, so that addresses
            // and descriptors stay in uniform registers, where the MMAs want
            // them (8192 tokens 4096 -> 11008, 4 bits: 114.4 us with one lane
            // in the loop, 111 so).
            const bool leader = elect_lane();
            int s = 0, buf = 0, it = 0;
            uint32_t ph = 0;
            bool ok = true, ready = false;
            const uint64_t ad0 = sw128_desc(sbase), bd0 = sw128_desc(sbase + L::off_x);
            auto spin = [&](uint64_t *bar, uint32_t phase) {
                return __all_sync(0xffffffffu, pair_spin(bar, phase, wait_limit, &abort_flag)) != 0;
            };
            for (long long i = pair; i < tiles && ok; i += pairs, ++it) {
                const uint32_t d = tmem + (it & 1) * L::kCol1;
                // The epilogue frees what this accumulator shares with the
                // previous tile's first of all; without shared columns the
                // one two tiles back has to be free.
                const int before = it - (shared ? 1 : 2);
                if (before >= 0) ok = spin(&acc_free[before & 1], (before >> 1) & 1);
                for (int c = 0; c < chunks && ok; ++c) {
                    if (!ready) ok = spin(&full[s], ph);
                    if (!ok) break;
                    mm_fence_after();
                    // (Descriptor addresses count 16 bytes and stay below 256 KB.)
                    const uint64_t ad = ad0 + (uint32_t)s * (L::stage >> 4), bd = bd0 + (uint32_t)s * (L::stage >> 4);
                    const uint32_t sw = tmem + L::kColScales + buf * L::kScaleCols, sx = sw + 4 * L::kScaleTiles;
                    const int kts = nkt - c * L::kScaleTiles;
                    if (leader) {
#pragma unroll
                        for (int m = 0; m < 4 * kSub; ++m) {
                            // 32 bytes of each row per MMA: with kX8 32 values and one
                            // scale byte, else 64 values and two.
                            const int sub = m / 4, q = m % 4, j = kX8 ? sub : m / 2, sf = kX8 ? q : 2 * (q % 2);
                            if (j == 0 || j < kts)
                                mx_mma<kX8, 2>(d, ad + sub * (kMmWBytes >> 4) + 2 * q,
                                               bd + sub * (L::x_block >> 4) + 2 * q,
                                               mx_idesc<kX8>(tile_tok, sf, 2 * kMmRows), sw + 4 * j, sx + L::kXCols * j,
                                               (c | m) != 0);
                        }
                        pair_commit(&empty[s]);
                    }
                    if (++s == L::kStages) s = 0, ph ^= 1u;
                    if (++buf == L::kScaleBufs) buf = 0;
                    ready = __all_sync(0xffffffffu, pair_test_wait(&full[s], ph));
                }
                if (leader) pair_commit(&acc_full[it & 1]);
                __syncwarp();
            }
            // Whatever was issued completes before tensor memory is freed.
            if (leader) {
                if (!ok) {
                    abort_flag = 1;
                    flag_timeout(status);
                }
                pair_commit(done);
            }
            __syncwarp();
            (void)mbar_wait_bounded(done, 0, wait_limit);
        }
        __syncwarp();
    } else if (warp < kPairEpiWarp) {
        // Scale warps: lane l of each lane quarter gets the words of rows l,
        // l + 32, l + 64 and l + 96, 16 adjacent bytes of a tile, as four
        // columns.  (tcgen05.cp does the same in one instruction, but for a
        // CTA pair each takes about 128 cycles of the tensor pipe, measured,
        // six per stage against four MMAs of about 128.)
        // Two groups of four take the stages in turn: an iteration lasts about
        // as long as a stage's MMAs.
        const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + L::kColScales;
        const uint32_t full0 = map_to_rank(smem_addr(full), 0);
        const int group = (warp - 2) >> 2;
        int n = 0;
        bool ok = true;
        for (long long i = pair; i < tiles && ok; i += pairs) {
            // Blocks of 32 tokens before the tile's first in its scale tile.
            const int skip = pair_tile(i, row_tiles, tok_tiles, tile_tok).tok0 % kMxTileRows / 32;
            for (int c = 0; c < chunks; ++c, ++n) {
                if ((n & 1) != group) continue;
                const int s = n % L::kStages, buf = n % L::kScaleBufs;
                ok = mbar_wait_abortable(&scales_in[s], (n / L::kStages) & 1, wait_limit, &abort_flag);
                if (n >= L::kScaleBufs) {
                    // The MMAs that last read this buffer.
                    const int m = n - L::kScaleBufs;
                    ok = ok && mbar_wait_abortable(&empty[m % L::kStages], (m / L::kStages) & 1, wait_limit,
                                                   &abort_flag);
                }
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) {
                        abort_flag = 1;
                        flag_timeout(status);
                    }
                    ok = false;
                    break;
                }
                mm_fence_after();
                const uint8_t *st = smem + s * L::stage + 16 * lane;
                const uint32_t col = t_lane + buf * L::kScaleCols;
                uint32_t ws[4 * L::kScaleTiles], xs[L::kXCols * L::kScaleTiles];
#pragma unroll
                for (int j = 0; j < L::kScaleTiles; ++j) {
                    auto put = [](uint32_t *to, uint4 f) { to[0] = f.x, to[1] = f.y, to[2] = f.z, to[3] = f.w; };
                    put(ws + 4 * j, *reinterpret_cast<const uint4 *>(st + L::off_sw + j * kMxTileBytes));
                    auto x_words = [&](int k) {
                        return k < x_tiles ? *reinterpret_cast<const uint4 *>(
                                                 st + L::off_sx + (k * L::kScaleTiles + j) * kMxTileBytes)
                                           : make_uint4(0u, 0u, 0u, 0u);
                    };
                    // The tile's first token goes to the first column: the
                    // MMA takes scales from a multiple of four columns on.
                    uint4 u = x_words(0), v = x_words(1);
                    if (skip) {
                        const uint4 w = kSub == 1 ? x_words(2) : make_uint4(0u, 0u, 0u, 0u);
                        if (skip == 1) {
                            u = make_uint4(u.y, u.z, u.w, v.x), v = make_uint4(v.y, v.z, v.w, w.x);
                        } else if (skip == 2) {
                            u = make_uint4(u.z, u.w, v.x, v.y), v = make_uint4(v.z, v.w, w.x, w.y);
                        } else {
                            u = make_uint4(u.w, v.x, v.y, v.z), v = make_uint4(v.w, w.x, w.y, w.z);
                        }
                    }
                    put(xs + L::kXCols * j, u);
                    if (kSub == 1) put(xs + L::kXCols * j + 4, v);
                }
                mm_st(col, ws);
                mm_st(col + 4 * L::kScaleTiles, xs);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                mm_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(full0 + 8 * s);
            }
        }
    } else {
        const int q = warp & 3, part = (warp - kPairEpiWarp) >> 2;  // lane quarter; every kPairEpi-th block of 32 tokens
        const uint32_t free_addr = map_to_rank(smem_addr(acc_free), 0);
        int it = 0;
        for (long long i = pair; i < tiles; i += pairs, ++it) {
            const PairTile t = pair_tile(i, row_tiles, tok_tiles, tile_tok);
            const bool ok = mbar_wait_abortable(&acc_full[it & 1], (it >> 1) & 1, wait_limit, &abort_flag);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) {
                    abort_flag = 1;
                    flag_timeout(status);
                }
                break;
            }
            mm_fence_after();
            const uint32_t col0 = tmem + ((uint32_t)(32 * q) << 16) + (it & 1) * L::kCol1;
            const int n = t.row0 + rank * kMmRows + 32 * q + lane;
            auto free_accumulator = [&]() {
                mm_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(free_addr + 8 * (it & 1));
            };
            // The shared columns are the last blocks of the first accumulator
            // and the first of the second, up to kPairEpi: one for each warp of a
            // quarter, which reads it before anything else, since the next
            // tile's MMAs wait for that.
            const int s0 = it & 1 ? 0 : blocks - shared;
            const int mine = s0 + (part + kPairEpi - s0 % kPairEpi) % kPairEpi;  // this warp's first block from s0 on
            const bool early = mine < s0 + shared;
            if (shared && !early) free_accumulator();
            bool first = early;
            for (int blk = early ? mine : part; blk < blocks;) {
                float v[32];
                mm_ld32(col0 + 32 * blk, v);
                if (first) free_accumulator();
                const int tok = t.tok0 + 32 * blk, count = min(32, T - tok);
                if (n < N && count > 0) {
                    const size_t at = (size_t)tok * N + n;
                    if (type == MxType::kF32)
                        store_column(static_cast<float *>(y) + at, N, count, v);
                    else if (type == MxType::kF16)
                        store_column(static_cast<__half *>(y) + at, N, count, v);
                    else
                        store_column(static_cast<__nv_bfloat16 *>(y) + at, N, count, v);
                }
                __syncwarp();
                blk = first ? part : blk + kPairEpi;
                first = false;
                if (early && blk == mine) blk += kPairEpi;
            }
            if (!shared) free_accumulator();
        }
    }
    mm_fence_before();
    __syncthreads();
    // The last commit arrives at both CTAs, and nothing else that the other
    // one does says that it has: each waits for it itself, or it could land
    // in the shared memory of the SM's next CTA.
    if (warp == 1) (void)mbar_wait_bounded(done, 0, wait_limit);
    __syncwarp();
    cluster_sync_all();  // neither CTA leaves while the other may signal it
    if (warp == 1) {
        mm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

PFN_cuTensorMapEncodeTiled_v12000 mm_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Map of codes [rows][Kp] in boxes of 128 shared-memory bytes by `box_rows`:
// packed bytes, or (unpack) 4-bit values spread to 16 bytes per 16 values.
bool map_codes(CUtensorMap *m, const uint8_t *codes, int rows, int Kp, int bits, bool unpack, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = mm_encode_fn();
    if (!encode) return false;
    const cuuint64_t row_bytes = (cuuint64_t)Kp * bits / 8;
    const cuuint64_t dims[2] = {unpack ? (cuuint64_t)Kp : row_bytes, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode(m, unpack ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                  const_cast<uint8_t *>(codes), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kX8, int kTok>
cudaError_t launch_split(const LaunchCtx &c, MxType type, const MxMatmulArgs &a) {
    using L = MmLayout<kX8, kTok>;
    const int Kp = mx_padded(a.K);
    const int n_mma = a.T < kTok ? (a.T + 15) / 16 * 16 : kTok;
    alignas(64) CUtensorMap tm_w, tm_x;
    if (!map_codes(&tm_w, a.w_codes, a.N, Kp, 4, kX8, kMmRows) ||
        !map_codes(&tm_x, a.x_codes, a.T, Kp, a.x_bits, false, n_mma))
        return cudaErrorInvalidValue;
    auto kernel = mx_mm_split_kernel<kX8, kTok>;
    cudaError_t e = ensure_smem(kernel, L::total);
    if (e != cudaSuccess) return e;
    const int row_tiles = (a.N + kMmRows - 1) / kMmRows, tok_tiles = (a.T + kTok - 1) / kTok;
    const int stages = (Kp + L::kStageK - 1) / L::kStageK;
    const int S = mx_split(row_tiles, tok_tiles, a.T, stages, a.x_bits, c.num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(row_tiles * S, tok_tiles);
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = L::total;
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
    return cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_x, a.w_scales, a.x_scales, a.y, type, a.K, a.N, a.T, n_mma,
                              c.status, c.wait_limit, c.withhold);
}

template <bool kX8, int kSub>
cudaError_t launch_pair(const LaunchCtx &c, MxType type, const MxMatmulArgs &a, const MxPairTiles &g) {
    using L = PairLayout<kX8, kSub>;
    const int Kp = mx_padded(a.K);
    alignas(64) CUtensorMap tm_w, tm_x;
    if (!map_codes(&tm_w, a.w_codes, a.N, Kp, 4, kX8, kMmRows) ||
        !map_codes(&tm_x, a.x_codes, a.T, Kp, a.x_bits, false, g.tile_tok / 2))
        return cudaErrorInvalidValue;
    auto kernel = mx_mm_pair_kernel<kX8, kSub>;
    cudaError_t e = ensure_smem(kernel, L::total);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)g.row_tiles * g.tok_tiles;
    const int pairs = (int)(tiles < c.num_sms / 2 ? tiles : c.num_sms / 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = L::total;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, tm_w, tm_x, a.w_scales, a.x_scales, a.y, type, a.K, a.N, a.T, g.tile_tok,
                              g.x_tiles, g.row_tiles, g.tok_tiles, c.status, c.wait_limit, c.withhold);
}

template <bool kX8>
cudaError_t launch_mm_tokens(const LaunchCtx &c, MxType type, const MxMatmulArgs &a) {
    constexpr int kStageK = PairLayout<kX8, 1>::kStageK;
    const int stages = (mx_padded(a.K) + kStageK - 1) / kStageK;
    if (mx_use_pairs(a.T, a.N, stages, a.x_bits, c.num_sms)) {
        const MxPairTiles g = mx_pair_tiles(a.T, a.N, stages, a.x_bits, c.num_sms);
        return g.tile_tok <= kMxPairTwoBlocks ? launch_pair<kX8, 2>(c, type, a, g) : launch_pair<kX8, 1>(c, type, a, g);
    }
    if (a.T <= 16) return launch_split<kX8, 16>(c, type, a);
    if (a.T <= 64) return launch_split<kX8, 64>(c, type, a);
    return launch_split<kX8, 128>(c, type, a);
}

}  // namespace

cudaError_t launch_mx_matmul(const LaunchCtx &c, MxType type, const MxMatmulArgs &a) {
    return a.x_bits == 8 ? launch_mm_tokens<true>(c, type, a) : launch_mm_tokens<false>(c, type, a);
}

}  // namespace q4mm

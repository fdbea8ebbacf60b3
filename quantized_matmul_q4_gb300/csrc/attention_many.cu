// Attention over a paged MX cache for many rows a key/value head (sm_103a):
// prompts and chunks of them, tiles of 128 rows on tcgen05.
//
//   S[row][key]   = Q Kᵀ     128 x 128, fp16 in, fp32 in tensor memory
//   P             = 2^(...)  into tensor memory, over S
//   O[row][value] += P V     fp32 in tensor memory
//
// What bounds it is the chain of a tile's softmax and the issue slots that it
// shares with the other's.  256 rows by 128 keys take 2048 cycles of the tensor
// pipe (two products of 128 x 128 x D a tile), 1024 of the special functions, and
// some 2500 issue slots of each of the SM's four schedulers: a third the
// arithmetic of the scores, a fifth the codes of K and V, the rest what each of
// 16 warps does once a tile.  They take 4400 cycles.  So two tiles of 128
// rows share every dequantised key and value, and while the softmax of one is
// computed the pipe works on the other.  A prompt of 8192 tokens, 32 heads of
// 128, 8 bits: 536 us, 1025 TFLOP/s (54% of the measured bf16 rate); 512 tokens over 8192,
// 8 key heads: 80 us, 828 TFLOP/s.  (Halves of a row that go by a maximum of their
// own, so that each waits for 64 keys' products alone: 695 us; one warp a quarter
// with whole rows has no exchange, but too few warps.)
//
// Warps of a CTA:
//   softmax  eight a tile: a thread has half of a row's 128 scores, so that
//            they stay in its registers (a warp reaches only its own quarter of the lanes
//            of tensor memory).  Maximum, shared with the other half's thread
//            through shared memory, exponentials, P, and, where the maximum
//            has grown by more than 8, O rescaled.
//   dequant  four, 32 neighbouring tokens of a tile each: codes to fp16 in
//            shared memory, rows of 128 bytes in the 128-byte swizzle.  V lies
//            like K, token by token: it is the product's B operand with the
//            values (N) contiguous.  The power of two taken out (see
//            attention.cuh) is one for those 32 tokens, and goes to the
//            softmax beside them.
//   copy     one: the codes and scales of 16 neighbouring tokens of a head are
//            one run of a page, hence one bulk copy each, a lane each.
//   issue    one warp, one elected lane: S of both tiles, then in turn P V of
//            one tile and S of its next keys.
// S of the next keys is written over P by an instruction issued after the one
// that reads P: instructions of one thread run in order.  A tile's softmax
// starts when its S is complete, hence also the P V before it, so it may
// rescale O; P V of these keys waits for its P.
//
// fp32 queries take two fp16 terms each for Q and P, and one tile of rows.
//
// Keys may be split over a cluster; the parts' sums are joined in rank order.
#include <cstdint>

#include "attention.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "sync.cuh"

namespace q4mm {

namespace {

// kDP: the head's values rounded up to 64 or 128; kTiles x kNP: tiles of 128
// rows and fp16 terms of a query value, 2 x 1 or 1 x 2.
template <int kBits, int kDP, int kTiles, int kNP>
struct ManyLayout {
    static constexpr int kSoftmaxWarps = 8 * kTiles, kDequantWarps = 4;
    static constexpr int kIssueWarp = kSoftmaxWarps + kDequantWarps, kCopyWarp = kIssueWarp + 1;
    static constexpr int kWarps = kIssueWarp + 4;
    static constexpr int kThreads = 32 * kWarps;
    // 24 warps have 80 registers each; of an SM quarter's 6 x 80 the softmax
    // takes 4 x 96, dequant 56, issue and copy 40.
    static constexpr bool kSplitRegs = kTiles == 2;
    static constexpr uint32_t kSlab = kManyKeys * kDP * 2;             // 128 rows of Q, K or V
    static constexpr int kSlots = kDP == 64 ? 6 : 3;                   // of the ring of K and V
    static constexpr int kMeta = 4;                                    // tiles whose powers are kept
    static constexpr uint32_t kCodes = kManyKeys * kDP * kBits / 8;    // codes of 128 rows
    static constexpr int kCodeSlots = kDP == 128 && kBits == 8 ? 3 : 4;
    static constexpr uint32_t off_ring = 2 * kSlab;
    static constexpr uint32_t off_codes = off_ring + kSlots * kSlab;
    static constexpr uint32_t off_scales = off_codes + kCodeSlots * kCodes;  // of K and V, 512 bytes each, two tiles
    static constexpr uint32_t off_end = off_scales + 2 * 1024;
    // The sums, where the operands were.
    static constexpr int kPitch = kDP + 4;
    static constexpr uint32_t total = off_end + 1024;  // the base is rounded up to 1024 bytes
    static_assert(total + 15 * 1024 <= kSmShared - kCtaSharedExtra, "room for ManyShared");
    static_assert(256 * 48 <= kCodeSlots * kCodes, "room for a RowOut a row");
    static_assert(kTiles * kNP == 2 && kTiles * 128 * kPitch * 4 <= off_codes, "");
    static_assert(kSmShared - total - kCtaSharedExtra < kHalfTmemShared, "takes all of tensor memory");
    // Powers of tile i + kMeta are written when S of tile i + kMeta - kSlots / 2 is done, after P of tile i.
    static_assert(kMeta > kSlots / 2, "");
    // Tensor memory: S (and P over it), second terms of P, O.
    static constexpr uint32_t col_s(int t) { return 128 * t; }
    // P's 16 keys k: over the S of the same half of the keys.
    static __device__ constexpr uint32_t col_p(int k) { return k / 4 * 64 + 8 * (k % 4); }
    static constexpr uint32_t kColLow = 128;  // kNP == 2, kTiles == 1
    static constexpr uint32_t col_o(int t) { return 256 + kDP * t; }
    // Tensor-core sums drop what falls below their last bit, so that long ones
    // fall short (one of 7500 keys by 1.6e-5 of its value, 940 steps of 16).
    // With fp32 outputs they are therefore taken every two tiles of keys, 32
    // steps, and added up by fp32 additions in other columns.  (16-bit outputs:
    // kChainF16 and kChainBf16 bound their steps, by more CTAs or by this form.)
    static constexpr int kDrain = kNP == 2 ? 2 : 0;
    static constexpr uint32_t kColSum = 384;
};

struct ManyShared {
    uint64_t ring_full[6], ring_free[6], code_full[4], code_free[4], meta_full[4], s_full[2], p_full[2], q_full, done,
        dequant_done;
    int kref[4][4], vref[4][4];  // powers of a tile's 32-token groups,
    int wide[4][4];              // or whether each token has its own:
    short krefs[4][128], vrefs[4][128];
    uint32_t valid[4];           // a tile's 16-token groups that were copied
    float top[2][2][256];        // a tile's maxima, of both halves
    int power[256];              // of two, taken out of a query row
    float m[256], l[2][256];
    uint4 mults[2][128];         // of a tile's tokens of K and V: each block's multiplier as two fp16
    int nan_from[4];
    uint32_t tmem;
    int abort;
    int spoilt, suspect;  // values that the sums cannot take were met; NaN among a row's values
};

static_assert(sizeof(ManyShared) <= 15 * 1024, "");

// What a row's output is made of: how much each CTA's sums count, the
// reciprocal of the sum, blocks that are NaN, its place in y.
struct RowOut {
    float by[kMaxSplit];
    float scale;
    int nan;
    long long at;
};

__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// Columns of this thread's lane, there when this returns.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// 64 columns, by two loads.
__device__ __forceinline__ void tc_ld64(uint32_t taddr, uint32_t (&a)[32], uint32_t (&b)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31 "
        "}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, "
        "%52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63 "
        "}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
          "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]),
          "=r"(a[15]), "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]),
          "=r"(a[22]), "=r"(a[23]), "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]),
          "=r"(a[29]), "=r"(a[30]), "=r"(a[31]), "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]),
          "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]),
          "=r"(b[13]), "=r"(b[14]), "=r"(b[15]), "=r"(b[16]), "=r"(b[17]), "=r"(b[18]), "=r"(b[19]),
          "=r"(b[20]), "=r"(b[21]), "=r"(b[22]), "=r"(b[23]), "=r"(b[24]), "=r"(b[25]), "=r"(b[26]),
          "=r"(b[27]), "=r"(b[28]), "=r"(b[29]), "=r"(b[30]), "=r"(b[31])
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Shared-memory operands in the 128-byte swizzle: 8 rows of 128 bytes are
// 1024.  K-major (Q, K: rows are M or N, 64 values of the head a row): groups
// of 8 rows 1024 bytes apart.  N-major (V: rows are keys, 64 of the N values a
// row): groups of 8 keys 1024 bytes apart, the next 64 values `next` bytes on.
__device__ __forceinline__ uint64_t k_major_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
__device__ __forceinline__ uint64_t n_major_desc(uint32_t saddr, uint32_t next) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(next >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
// kind::f16 with fp16 operands and fp32 sums, M = 128; B is N-major or K-major.
__device__ __forceinline__ constexpr uint32_t f16_idesc(int n, bool b_n_major) {
    return 1u << 4 | (b_n_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// Bulk copy from global to shared memory (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_copy(uint32_t to, const void *from, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                 "l"(from), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ bool elect_lane() {
    uint32_t mine;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(mine));
    return mine != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// kEach neighbouring values as they lie in memory: floats (kNP == 2), or pairs of 16 bits.
template <int kEach, int kNP>
struct RawRow {
    uint32_t w[kEach * kNP / 2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (uint32_t &x : w) x = 0u;
    }
    __device__ __forceinline__ void load(const void *p, long long at, bool vec, MxType type) {
        constexpr int kWords = kEach * kNP / 2;
        if (kNP == 2 && type != MxType::kF32) {  // 16-bit rows as fp32 ones
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = __float_as_uint(wide_value(p, type, at + i));
        } else if (vec) {
            const char *q = static_cast<const char *>(p) + at * (2 * kNP);
            if constexpr (kWords == 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(q);
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
            } else if constexpr (kWords == 2) {
                const uint2 u = *reinterpret_cast<const uint2 *>(q);
                w[0] = u.x, w[1] = u.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t *>(q);
            }
        } else if constexpr (kNP == 2) {
            const uint32_t *q = static_cast<const uint32_t *>(p) + at;
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = q[i];
        } else {
            const uint16_t *q = static_cast<const uint16_t *>(p) + at;
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = q[2 * i] | (uint32_t)q[2 * i + 1] << 16;
        }
    }
    __device__ __forceinline__ void values(MxType type, float (&v)[kEach]) const {
        if constexpr (kNP == 2) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kEach / 2; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[2 * i] = type == MxType::kF16 ? f.x : __uint_as_float(w[i] << 16);
                v[2 * i + 1] = type == MxType::kF16 ? f.y : __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
};

// The softmax warps' share of the CTA's rows, over its keys, by plain_row, to where the sums lie.  (A function of its
// own that finds rows and keys anew, so that the kernel holds nothing for it.)
template <int kBits, int kDP, int kTiles, int kNP>
__device__ __noinline__ void many_plain(const MxAttentionArgs &a, ManyShared &sh, uint32_t base, int group, long long tiles) {
    using L = ManyLayout<kBits, kDP, kTiles, kNP>;
    const int lane = threadIdx.x & 31, S = (int)cluster_size(), rank = (int)cluster_rank();
    const unsigned item = blockIdx.x / (unsigned)S;
    const RowTile tile = row_tile(a.batch, tiles - 1 - item / (unsigned)a.cache.heads, group, 128 * kTiles, a.tokens);
    const int keys = min(keys_of(tile, tile.first + tile.rows - 1, group, a.causal), table_keys(a.batch.width, a.cache.page));
    const int all = (keys + kManyKeys - 1) / kManyKeys, j0 = (int)((unsigned)all * (unsigned)rank / (unsigned)S),
              j1 = (int)((unsigned)all * (unsigned)(rank + 1) / (unsigned)S);
    for (int r = threadIdx.x / 32; r < tile.rows; r += L::kSoftmaxWarps) {
        const PlainSums p = plain_row<kBits>(a, tile, tile.first + r, group, (int)(item % (unsigned)a.cache.heads), keys,
                                             kManyKeys / 16 * j0, kManyKeys / 16 * j1, 1);
        // M of the largest value's size, as in the kernel's own sums, with which these are joined.  (Of two
        // CTAs' keys, values 2^180 below the others may be lost.)
        float top = fmaxf(fmaxf(fabsf(p.o.x), fabsf(p.o.y)), fmaxf(fabsf(p.o.z), fabsf(p.o.w)));
#pragma unroll
        for (int x = 1; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, kVrefMin), kVrefMax);
        const float by = pow2(-e);
        if (lane == 0) {
            sh.m[r] = isnan(p.m) ? -INFINITY : p.m + kPShift + (float)e;
            sh.l[0][r] = isnan(p.m) ? p.m : p.m == -INFINITY ? 0.f : by, sh.l[1][r] = 0.f;
        }
        if (4 * lane < kDP)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(base + (r * L::kPitch + 4 * lane) * 4),
                         "f"(p.o.x * by), "f"(p.o.y * by), "f"(p.o.z * by), "f"(p.o.w * by)
                         : "memory");
    }
}

template <int kBits, int kDP, int kTiles, int kNP>
__global__ void __launch_bounds__(ManyLayout<kBits, kDP, kTiles, kNP>::kThreads, 1)
    mx_attention_many_kernel(const __grid_constant__ MxAttentionArgs a, const int group, const long long tiles,
                             const long long wait_limit, const int withhold) {
    using L = ManyLayout<kBits, kDP, kTiles, kNP>;
    constexpr int kRows = 128 * kTiles;
    constexpr uint32_t kHalf = kManyKeys * 128;  // bytes of 64 values of 128 rows
    extern __shared__ uint8_t raw[];
    __shared__ ManyShared sh;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    // (By a shuffle, so that the compiler knows it to be one a warp, here and below.)
    auto uniform = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
    const int lane = threadIdx.x & 31, warp = uniform(threadIdx.x / 32);
    const int S = (int)cluster_size(), rank = (int)cluster_rank();
    const int D = a.cache.D;
    volatile int *abort = &sh.abort;

    pdl_wait();
    // (Divisions of 32 bits here: ones of 64 take a hundred instructions each.)
    const unsigned item = blockIdx.x / (unsigned)S;
    const int head = (int)(item % (unsigned)a.cache.heads);
    // (The last tiles first: with a causal mask they see the most keys.)
    const RowTile tile = row_tile(a.batch, tiles - 1 - item / (unsigned)a.cache.heads, group, kRows, a.tokens);
    if (tile.rows == 0) return;  // with the whole cluster

    // Keys that each tile of 128 rows sees, in tiles of 128, and this CTA's share of them.
    const int room = table_keys(a.batch.width, a.cache.page);
    int cnt[2] = {0, 0}, keys = 0;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int rows = min(max(tile.rows - 128 * t, 0), 128);
        int n = rows ? keys_of(tile, tile.first + 128 * t + rows - 1, group, a.causal) : 0;
        if (n > room) {
            if (threadIdx.x == 0) atomicOr(a.status, kStatusIndex);
            n = room;
        }
        keys = max(keys, n);
        cnt[t] = (n + kManyKeys - 1) / kManyKeys;
    }
    const int all = max(cnt[0], cnt[1]);
    // (A tile is 128 keys: all · S is below 2^28.)
    const int j0 = (int)((unsigned)all * (unsigned)rank / (unsigned)S), j1 = (int)((unsigned)all * (unsigned)(rank + 1) / (unsigned)S);
    cnt[0] = uniform(max(min(cnt[0], j1) - j0, 0)), cnt[1] = uniform(max(min(cnt[1], j1) - j0, 0));
    const int steps = max(cnt[0], cnt[1]);

    if (warp == L::kIssueWarp) {
        if (lane == 0) {
            for (int i = 0; i < L::kSlots; ++i) mbar_init(&sh.ring_full[i], L::kDequantWarps), mbar_init(&sh.ring_free[i], 1);
            for (int i = 0; i < L::kCodeSlots; ++i)
                mbar_init(&sh.code_full[i], 1), mbar_init(&sh.code_free[i], L::kDequantWarps);
            for (int i = 0; i < L::kMeta; ++i) mbar_init(&sh.meta_full[i], L::kDequantWarps);
            for (int i = 0; i < 2; ++i) mbar_init(&sh.s_full[i], 1), mbar_init(&sh.p_full[i], 8);
            mbar_init(&sh.q_full, L::kSoftmaxWarps), mbar_init(&sh.done, 1);
            mbar_init(&sh.dequant_done, L::kDequantWarps);
            fence_mbar_init();
            sh.abort = 0, sh.spoilt = 0, sh.suspect = 0;
            for (int i = 0; i < 4; ++i) sh.nan_from[i] = kNever;
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // Every warp ends by these, in its own role, so that no role holds registers for what another does afterwards.
    auto meet = [&]() {  // the CTA's sums, and its cluster's, are in shared memory
        __syncwarp();
        named_bar_sync(0, L::kThreads);
        if (cluster_size() > 1) cluster_sync_all();
    };
    auto leave = [&]() {  // no CTA leaves while another reads its sums
        __syncwarp();
        if (cluster_size() > 1)
            cluster_sync_all();
        else
            named_bar_sync(0, L::kThreads);
    };
    auto give_up = [&]() {
        if (lane == 0) {
            *abort = 1;
            flag_timeout(a.status);
        }
    };

    if (warp < L::kSoftmaxWarps) {
        // ---- softmax ----
        if constexpr (L::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
        const int t = warp / 8, side = warp / 4 % 2, quarter = warp % 4;
        const int mine = 128 * t + 32 * quarter + lane;  // this thread's row of the CTA's
        {
            // Query rows to fp16, each by a power of two of its own, 16 a warp,
            // the loads of 8 under way at once (one after the other they took 6 us).
            constexpr int kEach = kDP / 32, kAtOnce = 8;
            const uint32_t slab = base + t * kNP * L::kSlab;
            const int d = lane * kEach;
            const uint32_t col = (d / 64) * kHalf + (d % 8) * 2;
            const int first = 128 * t + 32 * quarter + 16 * side;  // of the tile's
            int tok = (tile.first + first) / group, row_head = (tile.first + first) % group;
#pragma unroll 1
            for (int b = 0; b < 16; b += kAtOnce) {
                RawRow<kEach, kNP> rows[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    rows[i].zero();
                    if (first + b + i < tile.rows && d < D)
                        rows[i].load(a.q, (long long)(tile.start + tok) * a.q_token + (long long)(head * group + row_head) * a.q_head + d,
                                     a.vec, a.type);
                    if (++row_head == group) row_head = 0, ++tok;
                }
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const int r = 32 * quarter + 16 * side + b + i;  // row of the slab
                    float v[kEach];
                    rows[i].values(a.type, v);
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < kEach; ++k) top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
                    top = __reduce_max_sync(0xFFFFFFFFu, top);
                    // 2^(141 - e) puts a largest value of biased exponent e at 2^14; not where it is infinite or NaN.
                    const int e = top >= 0x7F800000u ? 141 : max((int)(top >> 23), 15);
                    if (lane == 0) sh.power[128 * t + r] = e - 141;
                    const float mult = __int_as_float((268 - e) << 23);
                    const uint32_t at = slab + col + r * 128 + (((d % 64) / 8) ^ (r & 7)) * 16;
                    uint32_t hi[kEach / 2];
#pragma unroll
                    for (int k = 0; k < kEach / 2; ++k) hi[k] = half2_of(v[2 * k] * mult, v[2 * k + 1] * mult);
                    if constexpr (kEach == 4)
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(hi[0]), "r"(hi[1]) : "memory");
                    else
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(hi[0]) : "memory");
                    if constexpr (kNP == 2) {
                        uint32_t lo[kEach / 2];
#pragma unroll
                        for (int k = 0; k < kEach / 2; ++k) {
                            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi[k]));
                            lo[k] = half2_of(v[2 * k] * mult - b.x, v[2 * k + 1] * mult - b.y);
                        }
                        if constexpr (kEach == 4)
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + L::kSlab), "r"(lo[0]), "r"(lo[1])
                                         : "memory");
                        else
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + L::kSlab), "r"(lo[0]) : "memory");
                    }
                }
            }
        }
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);
        bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_prompt(&sh.q_full, 0, wait_limit, abort));

        const int power = sh.power[mine];
        const int sees = mine < tile.rows ? keys_of(tile, tile.first + mine, group, a.causal) : 0;
        const float c0 = a.scale * kLog2e;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t s_at = tmem + lanes + L::col_s(t) + 64 * side, o_at = tmem + lanes + L::col_o(t) + kDP / 2 * side;
        constexpr int kDrain = L::kDrain;
        const uint32_t sum_at = tmem + lanes + L::kColSum + kDP / 2 * side;
        float M = -INFINITY, l = 0.f;
        const int n = cnt[t];
        // Keys of this half, from the CTA's first on, that every row of the warp sees.
        const int full = __reduce_min_sync(0xFFFFFFFFu, sees - kManyKeys * j0 - 64 * side);
        bool go = true;  // the two warps of a quarter leave together, also after a time-out
        for (int i = 0; i < n && go; ++i) {
            const int mi = i % L::kMeta;
            ok = ok && mbar_wait_prompt(&sh.s_full[t], i & 1, wait_limit, abort) &&
                 mbar_wait_prompt(&sh.meta_full[mi], (i / L::kMeta) & 1, wait_limit, abort);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) give_up();
            tc_fence_after();
            const bool partial = kManyKeys * i + 64 > full;
            const int lim = partial ? sees - kManyKeys * (j0 + i) - 64 * side : 64;  // these keys below it are seen
            uint32_t x[2][32];
            tc_ld64(s_at, x[0], x[1]);
            float factor[2], vref[2], top = -INFINITY;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                factor[g] = c0 * pow2(power + sh.kref[mi][2 * side + g]), vref[g] = (float)sh.vref[mi][2 * side + g];
                if (sh.wide[mi][2 * side + g]) {
                    const short *kr = &sh.krefs[mi][64 * side + 32 * g], *vr = &sh.vrefs[mi][64 * side + 32 * g];
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        x[g][k] = __float_as_uint(fmaf(__uint_as_float(x[g][k]), c0 * pow2(power + kr[k]), (float)vr[k]));
                    factor[g] = 1.f, vref[g] = 0.f;
                }
                float m = -INFINITY, m2 = -INFINITY;
                if (partial) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (k < lim - 32 * g) m = fmaxf(m, __uint_as_float(x[g][k]));
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        m = max3(m, __uint_as_float(x[g][k]), __uint_as_float(x[g][k + 1]));
                        m2 = max3(m2, __uint_as_float(x[g][k + 2]), __uint_as_float(x[g][k + 3]));
                    }
                    m = fmaxf(m, m2);
                }
                top = fmaxf(top, m == -INFINITY ? -INFINITY : fmaf(m, factor[g], vref[g]));
            }
            // The other half's maximum (NaN: it gives up).  Both threads of a row
            // hold the same M.
            sh.top[i & 1][side][mine] = ok ? top : __int_as_float(0x7FC00000);
            named_bar_sync(1 + 4 * t + quarter, 64);
            const float other = sh.top[i & 1][side ^ 1][mine];
            go = ok && !isnan(other);
            top = fmaxf(top, other);
            float grown = 1.f;
            if (__any_sync(0xFFFFFFFFu, top > M + kPSlack)) {
                const float now = fmaxf(M, top), by = M == -INFINITY ? 0.f : ex2(M - now);
                M = now, l *= by;
                if (kDrain > 0) grown = by;
                if (kDrain == 0 && i > 0) {
#pragma unroll 1
                    for (int k = 0; k < kDP / 2; k += 16) {
                        uint32_t o[16];
                        tc_ld16(o_at + k, o);
#pragma unroll
                        for (int z = 0; z < 16; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * by);
                        tc_st16(o_at + k, o);
                    }
                }
            }
            if constexpr (kDrain > 0) {
                const bool drain = i > 0 && i % kDrain == 0;
                if (i > 0 && (drain || __any_sync(0xFFFFFFFFu, grown != 1.f))) {
#pragma unroll 1
                    for (int k = 0; k < kDP / 2; k += 16) {
                        uint32_t o[16], sums[16];
                        tc_ld16(o_at + k, o);
                        if (i > kDrain) {
                            tc_ld16(sum_at + k, sums);
                        } else {
#pragma unroll
                            for (int z = 0; z < 16; ++z) sums[z] = 0u;
                        }
#pragma unroll
                        for (int z = 0; z < 16; ++z) {
                            const float x = __uint_as_float(o[z]), y = __uint_as_float(sums[z]);
                            sums[z] = __float_as_uint((drain ? x + y : y) * grown), o[z] = __float_as_uint(x * grown);
                        }
                        if (!drain) tc_st16(o_at + k, o);
                        if (drain || i > kDrain) tc_st16(sum_at + k, sums);
                    }
                }
            }
            const float shift = (M == -INFINITY ? 0.f : M) - kPShift;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float2 f2 = make_float2(factor[g], factor[g]);
                const float2 b2 = make_float2(vref[g] - shift, vref[g] - shift);
                float2 sum = make_float2(0.f, 0.f);
                uint32_t p[16], low[16];
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    float2 e = ffma2(make_float2(__uint_as_float(x[g][k]), __uint_as_float(x[g][k + 1])), f2, b2);
                    x[g][k] = __float_as_uint(ex2(e.x)), x[g][k + 1] = __float_as_uint(ex2(e.y));
                }
                if (partial) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (k >= lim - 32 * g) x[g][k] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const float2 e = make_float2(__uint_as_float(x[g][k]), __uint_as_float(x[g][k + 1]));
                    sum = __fadd2_rn(sum, e);
                    p[k / 2] = half2_of(e.x, e.y);
                    if constexpr (kNP == 2) {
                        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&p[k / 2]));
                        low[k / 2] = half2_of(e.x - b.x, e.y - b.y);
                    }
                }
                if (sh.wide[mi][2 * side + g]) {
                    const short *vr = &sh.vrefs[mi][64 * side + 32 * g];
#pragma unroll
                    for (int k = 0; k < 32; ++k) l = fmaf(__uint_as_float(x[g][k]), pow2(-vr[k]), l);
                } else {
                    l = fmaf(sum.x + sum.y, pow2(-(int)vref[g]), l);
                }
                tc_st16(s_at + 16 * g, p);
                if constexpr (kNP == 2) tc_st16(tmem + lanes + L::kColLow + 32 * side + 16 * g, low);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[t]);
        }
        if (!go) give_up();
        // The sums to shared memory, where the operands were.
        ok = mbar_wait_prompt(&sh.done, 0, wait_limit, abort) &&
             mbar_wait_prompt(&sh.dequant_done, 0, wait_limit, abort);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
            give_up();
        } else {
            tc_fence_after();
            float any = 0.f;
            sh.m[mine] = M, sh.l[side][mine] = l;
            const uint32_t to = base + (mine * L::kPitch + kDP / 2 * side) * 4;
#pragma unroll
            for (int k = 0; k < kDP / 2; k += 32) {
                uint32_t o[32];
                if (n > 0) {
                    tc_ld32(o_at + k, o);
                    if (kDrain > 0 && n > kDrain) {
                        uint32_t sums[32];
                        tc_ld32(sum_at + k, sums);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            o[x] = __float_as_uint(__uint_as_float(o[x]) + __uint_as_float(sums[x]));
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = 0u;
                }
#pragma unroll
                for (int x = 0; x < 32; x += 4) {
                    any += __uint_as_float(o[x]) + __uint_as_float(o[x + 1]) + (__uint_as_float(o[x + 2]) + __uint_as_float(o[x + 3]));
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + 4 * (k + x)), "r"(o[x]),
                                 "r"(o[x + 1]), "r"(o[x + 2]), "r"(o[x + 3])
                                 : "memory");
                }
            }
            tc_fence_before();
            if (isnan(any)) sh.suspect = 1, sh.top[0][side][mine] = any;
        }
        // A code of v that is NaN reaches rows that do not see it here: they have NaN among their values, but not in their sum.
        named_bar_sync(9, 32 * L::kSoftmaxWarps);
        if (sh.suspect) {
            if (isnan(sh.top[0][side][mine]) && !isnan(sh.l[0][mine] + sh.l[1][mine])) sh.spoilt = 1;
            named_bar_sync(9, 32 * L::kSoftmaxWarps);
        }
        if (sh.spoilt && !*abort) many_plain<kBits, kDP, kTiles, kNP>(a, sh, base, group, tiles);
        meet();
        {
            // Each CTA of the cluster joins and writes its share of the rows:
            // first a thread a row, by how much each CTA's sums count.
            const int parts = (int)cluster_size(), part = (int)cluster_rank();
            constexpr int kThreads = 32 * L::kSoftmaxWarps, kQuads = kDP / 4;
            const int r0 = tile.rows * part / parts, here = tile.rows * (part + 1) / parts - r0;
            RowOut *out = reinterpret_cast<RowOut *>(raw + (base - smem_addr(raw)) + L::off_codes);
            const uint32_t m_at = smem_addr(sh.m), l_at = smem_addr(sh.l), n_at = smem_addr(sh.nan_from);
            if ((int)threadIdx.x < here) {
                const int r = r0 + threadIdx.x, row = tile.first + r, tok = row / group, sees = keys_of(tile, row, group, a.causal);
                float m[kMaxSplit], l[kMaxSplit], top = -INFINITY, ls = 0.f;
                RowOut o;
                o.nan = 0;
#pragma unroll
                for (int s = 0; s < kMaxSplit; ++s) {
                    m[s] = -INFINITY, l[s] = 0.f;
                    if (s >= parts) continue;
                    m[s] = ld_cluster_f32(map_to_rank(m_at + 4 * r, s));
                    l[s] = ld_cluster_f32(map_to_rank(l_at + 4 * r, s)) + ld_cluster_f32(map_to_rank(l_at + 4 * (256 + r), s));
#pragma unroll
                    for (int b = 0; b < kDP / kMxBlock; ++b)
                        o.nan |= (__float_as_int(ld_cluster_f32(map_to_rank(n_at + 4 * b, s))) < sees) << b;
                    top = fmaxf(top, m[s]);
                }
#pragma unroll
                for (int s = 0; s < kMaxSplit; ++s) {
                    o.by[s] = m[s] == -INFINITY ? 0.f : ex2(m[s] - top);
                    ls += m[s] == -INFINITY ? l[s] : o.by[s] * l[s];
                }
                // A row that sees nothing has no sum: zeros.  (One that does: scores of minus infinity alone, whose softmax is NaN.)
                o.scale = ls != 0.f ? 1.f / ls : sees > 0 ? __int_as_float(0x7FC00000) : 0.f;
                o.at = (long long)(tile.start + tok) * a.y_token + (long long)(head * group + row - tok * group) * a.y_head;
                out[threadIdx.x] = o;
            }
            named_bar_sync(9, kThreads);  // (1 to 8 are the halves' of a quarter)
            const int all_quads = *abort ? 0 : here * kQuads;
            if (parts == 1) {  // the sums lie here: four at a time
                const float *sums = reinterpret_cast<const float *>(raw + (base - smem_addr(raw)));
                for (int i = threadIdx.x; i < all_quads; i += 4 * kThreads) {
                    float4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = i + k * kThreads;
                        if (at < all_quads)
                            v[k] = *reinterpret_cast<const float4 *>(sums + at / kQuads * L::kPitch + 4 * (at % kQuads));
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = i + k * kThreads, d = 4 * (at % kQuads);
                        if (at >= all_quads || d >= D) continue;
                        const RowOut &o = out[at / kQuads];
                        const float by = o.by[0] * (o.nan >> (d / kMxBlock) & 1 ? __int_as_float(0x7FC00000) : o.scale);
                        store4(a.y, a.type, o.at + d, a.vec, make_float4(v[k].x * by, v[k].y * by, v[k].z * by, v[k].w * by));
                    }
                }
            }
            for (int i = parts == 1 ? all_quads : (int)threadIdx.x; i < all_quads; i += kThreads) {
                const int r = i / kQuads, d = 4 * (i % kQuads);
                if (d >= D) continue;
                const RowOut &o = out[r];
                const uint32_t from = base + 4 * ((r0 + r) * L::kPitch + d);
                float4 v[kMaxSplit];
#pragma unroll
                for (int s = 0; s < kMaxSplit; ++s)
                    if (s < parts) v[s] = ld_cluster_v4(map_to_rank(from, s));
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int s = 0; s < kMaxSplit; ++s) {
                    if (s >= parts) continue;
                    sum.x = fmaf(o.by[s], v[s].x, sum.x), sum.y = fmaf(o.by[s], v[s].y, sum.y);
                    sum.z = fmaf(o.by[s], v[s].z, sum.z), sum.w = fmaf(o.by[s], v[s].w, sum.w);
                }
                const float by = o.nan >> (d / kMxBlock) & 1 ? __int_as_float(0x7FC00000) : o.scale;
                store4(a.y, a.type, o.at + d, a.vec, make_float4(sum.x * by, sum.y * by, sum.z * by, sum.w * by));
            }
        }
        leave();
    } else if (warp < L::kSoftmaxWarps + L::kDequantWarps) {
        // ---- dequant ----
        if constexpr (L::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        constexpr int kLanes = kDP * kBits / 128;   // of 16 bytes a token
        constexpr int kEach = 32 / kLanes;          // tokens a load
        constexpr int kVals = 128 / kBits;          // values of a lane: 16 or 32
        const int w = warp - L::kSoftmaxWarps, c = lane % kLanes;
        const int half = c * kVals / 64, chunk = c * kVals % 64 / 8, block = c * kVals / kMxBlock;
        // Lanes of the second 64 values take another token, so that eight
        // lanes' stores meet in no bank.
        const int tok0 = (lane / kLanes) ^ (kDP == 64 ? 0 : kBits == 8 ? half : 2 * half);
        const bool in = c * kVals < D;
        const int blocks = D / kMxBlock, row_bytes = D * kBits / 8;
        // Where a lane's 16 bytes of token tok0 come from and go to; the next
        // tokens are kEach on.  (The swizzle of a row and the one kEach on
        // differ in bit 2 of the 16-byte chunk, or not at all.)
        const int r0 = 32 * w + tok0;
        const uint32_t from0 = base + L::off_codes + r0 * row_bytes + 16 * c;
        const uint32_t to0 = base + L::off_ring + half * kHalf + r0 * 128 + ((chunk ^ (r0 & 7)) * 16);
        const uint32_t mult0 = smem_addr(sh.mults) + r0 * 16 + block * 4;
        constexpr uint32_t kFlip = kEach == 4 ? 64 : 0;
        // A unit's codes (K of tile i: 2i, V: 2i + 1) to fp16 in its slot of the ring.
        auto put = [&](int unit) {
            uint32_t from = from0 + unit % L::kCodeSlots * L::kCodes, to = to0 + unit % L::kSlots * L::kSlab;
            uint32_t mult_at = mult0 + unit % 2 * 2048;
#pragma unroll 1
            for (int i = 0; i < kLanes; i += 2) {
                uint32_t word[2][4], m[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    word[j][0] = word[j][1] = word[j][2] = word[j][3] = 0u;
                    if (in)
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(word[j][0]), "=r"(word[j][1]), "=r"(word[j][2]), "=r"(word[j][3])
                                     : "r"(from + j * kEach * row_bytes)
                                     : "memory");
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(m[j]) : "r"(mult_at + j * kEach * 16) : "memory");
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t at = j ? (to + kEach * 128) ^ kFlip : to;
                    if constexpr (kBits == 8) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (16 * k)),
                                         "r"(half2_mul(half_e4m3x2(word[j][2 * k]), m[j])),
                                         "r"(half2_mul(half_e4m3x2_high(word[j][2 * k]), m[j])),
                                         "r"(half2_mul(half_e4m3x2(word[j][2 * k + 1]), m[j])),
                                         "r"(half2_mul(half_e4m3x2_high(word[j][2 * k + 1]), m[j]))
                                         : "memory");
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (16 * k)),
                                         "r"(half2_mul(half_e2m1x2<0>(word[j][k]), m[j])),
                                         "r"(half2_mul(half_e2m1x2<1>(word[j][k]), m[j])),
                                         "r"(half2_mul(half_e2m1x2<2>(word[j][k]), m[j])),
                                         "r"(half2_mul(half_e2m1x2<3>(word[j][k]), m[j]))
                                         : "memory");
                    }
                }
                from += 2 * kEach * row_bytes, to += 2 * kEach * 128, mult_at += 2 * kEach * 16;
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.code_free[unit % L::kCodeSlots]), mbar_arrive(&sh.ring_full[unit % L::kSlots]);
        };
        // This lane's token's multipliers, 2^(7 + exponent - ref): a NaN scale
        // infinite for K, whose zero codes make it NaN, and zero for V.
        auto put_mults = [&](const ScaleWord &s, int ref, bool is_v) {
            uint32_t m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = s.b[i] == 255 ? (is_v ? -127 : 128) : max(s.b[i] - 127 - ref, -127);
                const float f = __int_as_float((e + 127) << 23);
                m[i] = half2_of(f, f);
            }
            sh.mults[is_v][32 * w + lane] = make_uint4(m[0], m[1], m[2], m[3]);
        };
        // Codes of tokens that do not exist are zeros.
        auto clear = [&](int unit, uint32_t exists) {
            if (exists >> lane & 1) return;
            const uint32_t at = base + L::off_codes + unit % L::kCodeSlots * L::kCodes + (32 * w + lane) * row_bytes;
            for (int i = 0; i < row_bytes; i += 16)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + i), "r"(0) : "memory");
        };
        bool ok = true;
        auto ready = [&](int unit) {  // its codes are there, and its slot of the ring is free
            ok = mbar_wait_prompt(&sh.code_full[unit % L::kCodeSlots], (unit / L::kCodeSlots) & 1, wait_limit, abort) &&
                 (unit < L::kSlots || mbar_wait_prompt(&sh.ring_free[unit % L::kSlots], (unit / L::kSlots - 1) & 1,
                                                          wait_limit, abort));
            ok = __all_sync(0xFFFFFFFFu, ok);
            return ok;
        };
        for (int i = 0; i < steps; ++i) {
            if (!ready(2 * i)) break;
            const int mi = i % L::kMeta, left = keys - (kManyKeys * (j0 + i) + 32 * w);
            const uint32_t valid = sh.valid[mi] >> (2 * w);
            uint32_t exists = (valid & 1 ? 0xFFFFu : 0u) | (valid & 2 ? 0xFFFF0000u : 0u);
            if (left < 32) exists &= left > 0 ? (1u << left) - 1 : 0u;
            uint32_t ks = 0, vs = 0;
            if (exists >> lane & 1) {
                const uint32_t from = base + L::off_scales + i % 2 * 1024 + 4 * (32 * w + lane);
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(ks) : "r"(from) : "memory");
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vs) : "r"(from + 512) : "memory");
            }
            const ScaleWord sk(ks, blocks), sv(vs, blocks);
            const int kref = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)sk.top) - 134;
            const int vtop = (int)__reduce_max_sync(0xFFFFFFFFu, (unsigned)sv.top), vref = max(vtop - 134, kVrefMin);
            if (vref_passes(vtop)) sh.spoilt = 1;
            if (sv.nan) {  // NaN in v reaches the rows that see it, and no others
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (sv.b[b] == 255) atomicMin(&sh.nan_from[b], kManyKeys * (j0 + i) + 32 * w + lane);
            }
            int rk = kref, rv = vref;
            const bool wide = __any_sync(0xFFFFFFFFu, (sk.top != 0 && sk.top - 134 + kWide < kref) ||
                                                          (sv.top != 0 && sv.top - 134 + kWide < vref));
            if (wide) {
                if (sk.top != 0) rk = sk.top - 134;
                if (sv.top != 0) rv = max(sv.top - 134, kVrefMin);
                if (vref_passes(sv.top)) sh.spoilt = 1;
                sh.krefs[mi][32 * w + lane] = (short)rk, sh.vrefs[mi][32 * w + lane] = (short)rv;
                __syncwarp();
            }
            if (lane == 0) {
                sh.kref[mi][w] = kref, sh.vref[mi][w] = vref, sh.wide[mi][w] = wide;
                mbar_arrive(&sh.meta_full[mi]);
            }
            put_mults(sk, rk, false), put_mults(sv, rv, true);
#pragma unroll 1
            for (int v = 0; v < 2; ++v) {
                if (v && !ready(2 * i + 1)) break;
                if (exists != 0xFFFFFFFFu) clear(2 * i + v, exists);
                __syncwarp();
                put(2 * i + v);
            }
            if (!ok) break;
        }
        if (!ok) give_up();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.dequant_done);
        meet();
        leave();
    } else {
        if constexpr (L::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == L::kIssueWarp) {
            // ---- issue ----
            const bool leader = elect_lane();
            constexpr uint32_t kIdS = f16_idesc(kManyKeys, false), kIdO = f16_idesc(kDP, true);
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                ok = __all_sync(0xFFFFFFFFu, mbar_spin_abortable(bar, parity, wait_limit, abort));
                tc_fence_after();
                return ok;
            };
            auto scores = [&](int t, int i) {  // S of tile t and the CTA's keys i
                const uint64_t qd = k_major_desc(base + t * kNP * L::kSlab);
                const uint64_t kd = k_major_desc(base + L::off_ring + 2 * i % L::kSlots * L::kSlab);
                const bool last = t == 1 || cnt[1] <= i;  // no other tile wants K
                uint64_t *k_free = &sh.ring_free[2 * i % L::kSlots];
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kNP * kDP / 16; ++k) {
                        const int in = k % (kDP / 16);
                        const uint32_t at = in / 4 * (kHalf >> 4) + 2 * (in % 4);
                        // (Second terms first, while there is little to cut off.)
                        mma_ss(tmem + L::col_s(t), qd + (k < (kNP - 1) * kDP / 16 ? L::kSlab >> 4 : 0) + at, kd + at, kIdS, k != 0);
                    }
                    tc_commit(&sh.s_full[t]);
                    if (last) tc_commit(k_free);
                }
                __syncwarp();
            };
            auto outputs = [&](int t, int i) {
                const uint64_t vd = n_major_desc(base + L::off_ring + (2 * i + 1) % L::kSlots * L::kSlab, kHalf);
                const bool last = t == 1 || cnt[1] <= i;
                uint64_t *v_free = &sh.ring_free[(2 * i + 1) % L::kSlots];
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kNP * kManyKeys / 16; ++k) {
                        const int in = k % (kManyKeys / 16);
                        const uint32_t p_col = k < (kNP - 1) * kManyKeys / 16 ? L::kColLow + 8 * in : L::col_s(t) + L::col_p(in);
                        mma_ts(tmem + L::col_o(t), tmem + p_col, vd + (2048 >> 4) * in, kIdO, (L::kDrain > 0 ? i % L::kDrain : i) != 0 || k != 0);
                    }
                    if (last) tc_commit(v_free);
                }
                __syncwarp();
            };
            auto k_ready = [&](int i) { return wait(&sh.ring_full[2 * i % L::kSlots], (2 * i / L::kSlots) & 1); };
            auto v_ready = [&](int i) { return wait(&sh.ring_full[(2 * i + 1) % L::kSlots], ((2 * i + 1) / L::kSlots) & 1); };
            if (steps > 0 && wait(&sh.q_full, 0) && k_ready(0)) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    if (cnt[t] > 0) scores(t, 0);
                for (int i = 0; i < steps && ok; ++i) {
                    if (!v_ready(i)) break;
                    bool k_known = false;
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) {
                        if (i >= cnt[t]) continue;
                        if (!wait(&sh.p_full[t], i & 1)) break;
                        outputs(t, i);
                        if (i + 1 < cnt[t]) {
                            if (!k_known && !k_ready(i + 1)) break;
                            k_known = true;
                            scores(t, i + 1);
                        }
                    }
                }
            }
            if (!ok) give_up();
            // Whatever was issued completes before tensor memory is read or freed.
            if (leader) tc_commit(&sh.done);
            __syncwarp();
            if (!mbar_wait_bounded(&sh.done, 0, wait_limit)) outlast_copies();
            __syncwarp();
            meet();
            leave();
            if (*abort != 0) outlast_copies();
            tc_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
            return;
        }
        if (warp == L::kCopyWarp) {
            // ---- copy ----
            // Lane g + 8 · kind has the tile's tokens 16 g ..: kind 0 codes of K,
            // 1 and 2 scales of K and V, 3 codes of V.
            const int kind = lane / 8, g16 = lane % 8, row_bytes = D * kBits / 8, per_page = a.cache.page / 16;
            int piece = (8 * j0 + g16) / per_page, within = (8 * j0 + g16) % per_page;
            const uint8_t *from = kind == 0 ? a.cache.k_codes : kind == 1 ? a.cache.k_scales : kind == 2 ? a.cache.v_scales
                                                                                               : a.cache.v_codes;
            const int token_bytes = kind == 1 || kind == 2 ? 4 : row_bytes;
            const uint32_t bytes = 16 * token_bytes;
            auto next_page = [&](int i) {
                return i < steps && kManyKeys * (j0 + i) + 16 * g16 < keys ? page_of(a.batch, a.cache, tile.seq, piece, a.status)
                                                                           : -1;
            };
            int page = next_page(0), unit = 0;
            bool ok = true;
            auto slot_free = [&](int u) {
                if (u >= L::kCodeSlots)
                    ok = mbar_wait_prompt(&sh.code_free[u % L::kCodeSlots], (u / L::kCodeSlots - 1) & 1, wait_limit, abort);
                ok = __all_sync(0xFFFFFFFFu, ok);
                return ok;
            };
            const int held = withhold < 0 ? -1 : min(withhold, steps - 1);
            for (int i = 0; i < steps; ++i) {
                const uint8_t *at = from + (first_slot(a.cache, page, head) + 16 * within) * token_bytes;
                const bool mine = page >= 0;
                const uint32_t valid = __ballot_sync(0xFFFFFFFFu, mine) & 0xFF;
                const int groups = __popc(valid);
                within += 8 % per_page, piece += 8 / per_page;
                if (within >= per_page) within -= per_page, ++piece;
                page = next_page(i + 1);
                for (int v = 0; v < 2; ++v, ++unit) {
                    if (!slot_free(unit)) break;
                    uint64_t *full = &sh.code_full[unit % L::kCodeSlots];
                    if (lane == 0) {
                        sh.valid[i % L::kMeta] = valid;
                        if (i != held) mbar_arrive_expect_tx(full, groups * 16 * (row_bytes + (v ? 0 : 8)));
                    }
                    __syncwarp();
                    if (mine && i != held && (v ? kind == 3 : kind < 3)) {
                        const uint32_t to = kind == 1 || kind == 2
                                                ? base + L::off_scales + i % 2 * 1024 + (kind - 1) * 512 + 64 * g16
                                                : base + L::off_codes + unit % L::kCodeSlots * L::kCodes + 16 * g16 * row_bytes;
                        bulk_copy(to, at, bytes, full);
                    }
                }
                if (!ok) break;
            }
            if (!ok) {
                give_up();
                // No copy may still be writing shared memory at exit.
                outlast_copies();
            }
            __syncwarp();
        }
        meet();
        leave();
    }
}

template <int kBits, int kDP, int kTiles, int kNP>
cudaError_t launch_many(const LaunchCtx &c, const MxAttentionArgs &a, int S) {
    using L = ManyLayout<kBits, kDP, kTiles, kNP>;
    auto kernel = mx_attention_many_kernel<kBits, kDP, kTiles, kNP>;
    cudaError_t e = ensure_smem(kernel, L::total);
    if (e != cudaSuccess) return e;
    const int group = a.heads / a.cache.heads;
    const long long rows = (long long)a.tokens * group, tiles = rows / (128 * kTiles) + a.batch.seqs;
    const long long ctas = tiles * a.cache.heads * S;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(L::kThreads);
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
    return cudaLaunchKernelEx(&cfg, kernel, a, group, tiles, c.wait_limit, c.withhold);
}

template <int kBits, int kDP>
cudaError_t launch_type(const LaunchCtx &c, const MxAttentionArgs &a, int split, bool as_f32) {
    return as_f32 || a.type == MxType::kF32 ? launch_many<kBits, kDP, 1, 2>(c, a, split) : launch_many<kBits, kDP, 2, 1>(c, a, split);
}

}  // namespace

cudaError_t launch_mx_attention_many(const LaunchCtx &c, const MxAttentionArgs &a, int split, bool as_f32) {
    const bool narrow = a.cache.D <= 64;
    if (a.cache.bits == 4) return narrow ? launch_type<4, 64>(c, a, split, as_f32) : launch_type<4, 128>(c, a, split, as_f32);
    return narrow ? launch_type<8, 64>(c, a, split, as_f32) : launch_type<8, 128>(c, a, split, as_f32);
}

}  // namespace q4mm

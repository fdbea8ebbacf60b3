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
// as whole 512-byte tiles by plain bulk copies and are put into tensor memory
// with tcgen05.cp by the thread that issues the MMAs; copies and MMAs of one
// thread run in order.
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
    static_assert(kStages >= 2 && 2 * (total + 1024) <= 233472, "two CTAs per SM");
    static_assert(2 * kCols <= 512, "tensor memory of two CTAs");
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

// Block-scaled instruction descriptor: E8M0 scales, K-major operands, M = 128.
// sf: which byte of a scale column's 32-bit word the instruction starts at.
template <bool kX8>
__device__ __forceinline__ uint32_t mx_idesc(int n, int sf) {
    const uint32_t a_fmt = kX8 ? 5u : 1u;  // E2M1
    const uint32_t b_fmt = kX8 ? 0u : 1u;  // E4M3 or E2M1
    return (uint32_t)sf << 4 | a_fmt << 7 | b_fmt << 10 | (uint32_t)(n >> 3) << 17 | 1u << 23 |
           (uint32_t)(kMmRows >> 4) << 24 | (uint32_t)sf << 29;
}

template <bool kX8>
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t accumulate) {
    if constexpr (kX8) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    }
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

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Four consecutive n of one token, as the type asks; the aligned case is one
// store.
__device__ __forceinline__ void store_y4(void *y, MxType type, size_t at, int left, float4 v) {
    const float e[4] = {v.x, v.y, v.z, v.w};
    if (type == MxType::kF32) {
        float *p = static_cast<float *>(y) + at;
        if (left >= 4 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
            *reinterpret_cast<float4 *>(p) = v;
        } else {
            for (int i = 0; i < 4 && i < left; ++i) p[i] = e[i];
        }
    } else if (type == MxType::kF16) {
        __half *p = static_cast<__half *>(y) + at;
        for (int i = 0; i < 4 && i < left; ++i) p[i] = __float2half_rn(e[i]);
    } else {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(y) + at;
        for (int i = 0; i < 4 && i < left; ++i) p[i] = __float2bfloat16_rn(e[i]);
    }
}

// Up to 128 tokens per tile, K split over the CTAs of a cluster: rank r of S
// takes the stages [r·c/S, (r+1)·c/S) and puts its partial sums, [token][row],
// into its shared memory; rank s then adds the S partial sums of rows
// 4·(32·s/S) onwards in rank order, read over the cluster, and writes y, so
// the result does not depend on scheduling.
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

    if (threadIdx.x == 0) {
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
    if (warp == 1) {
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
    // Every operand may come from the previous kernel on the stream, the
    // weights too (a quantisation is a kernel like any other).
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            int c = 0;
            for (; c < chunks && !abort_flag; ++c) {
                const int s = c % L::kStages;
                if (c >= L::kStages &&
                    !mbar_wait_abortable(&empty[s], ((c / L::kStages) - 1) & 1, wait_limit, &abort_flag)) {
                    abort_flag = 1;
                    flag_timeout(status);
                    break;
                }
                if (c == withhold) continue;  // test only: this stage never arrives
                const int k0 = (c_lo + c) * L::kStageK, kt = (c_lo + c) * L::kScaleTiles;
                const uint32_t sbytes = (uint32_t)min(L::kScaleTiles, nkt - kt) * kMxTileBytes;
                uint8_t *st = smem + s * L::stage;
                const uint32_t sa = sbase + s * L::stage;
                mbar_arrive_expect_tx(&full[s], L::w_tx + n_mma * 128 + 2 * sbytes);
                const int c0 = kX8 ? k0 : k0 / 2;  // 8-bit codes and unpacked 4-bit ones in values, else bytes
                mm_tma_2d(sa, &tm_w, c0, row0, &full[s]);
                mm_tma_2d(sa + L::off_x, &tm_x, c0, tok0, &full[s]);
                bulk_g2s(st + L::off_sw, w_scales + ((size_t)row_tile * nkt + kt) * kMxTileBytes, sbytes, &full[s]);
                bulk_g2s(st + L::off_sx, x_scales + ((size_t)(tok0 / kMxTileRows) * nkt + kt) * kMxTileBytes, sbytes,
                         &full[s]);
            }
            // No copy may still be writing shared memory at exit.
            for (int i = max(0, c - L::kStages); i < c; ++i)
                if (i != withhold) (void)mbar_wait_bounded(&full[i % L::kStages], (i / L::kStages) & 1, wait_limit);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            for (int c = 0; c < chunks; ++c) {
                const int s = c % L::kStages;
                if (!mbar_spin_abortable(&full[s], (c / L::kStages) & 1, wait_limit, &abort_flag)) {
                    abort_flag = 1;
                    flag_timeout(status);
                    break;
                }
                mm_fence_after();
                const uint32_t sa = sbase + s * L::stage;
                const int kts = min(L::kScaleTiles, nkt - (c_lo + c) * L::kScaleTiles);
                for (int j = 0; j < kts; ++j) {
                    scale_to_tmem(tmem + L::kColSw + 4 * j, scale_desc(sa + L::off_sw + j * kMxTileBytes));
                    scale_to_tmem(tmem + L::kColSx + 4 * j, scale_desc(sa + L::off_sx + j * kMxTileBytes));
                }
                const uint64_t ad = sw128_desc(sa), bd = sw128_desc(sa + L::off_x);
                // 32 bytes of each row per MMA: with kX8 32 values and one scale
                // byte, else 64 values and two.
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int j = kX8 ? 0 : m / 2, sf = kX8 ? m : 2 * (m % 2);
                    if (j < kts)
                        mx_mma<kX8>(tmem, ad + 2 * m, bd + 2 * m, mx_idesc<kX8>(n_mma, sf), tmem + L::kColSw + 4 * j,
                                    tmem + L::kColSx + 4 * j, (c | m) != 0);
                }
                mm_commit(&empty[s]);
            }
            // Whatever was issued completes before tensor memory is read or freed.
            mm_commit(done);
            (void)mbar_wait_bounded(done, 0, wait_limit);
        }
        __syncwarp();
    }
    // (The producer and the issuer leave their branches through a reconverged
    // warp; every warp takes part from here on.)
    const bool ok = __syncthreads_and(mbar_wait_bounded(done, 0, wait_limit) ? 1 : 0) != 0 && !abort_flag;
    mm_fence_after();
    const int toks = min(kTok, T - tok0);
    float *part = reinterpret_cast<float *>(smem);  // [token][128 rows], over the ring
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
                for (int i = 0; i < 8; ++i) {
                    if (t + i >= toks) break;
                    const size_t at = (size_t)(tok0 + t + i) * N + n;
                    if (type == MxType::kF32)
                        static_cast<float *>(y)[at] = v[i];
                    else if (type == MxType::kF16)
                        static_cast<__half *>(y)[at] = __float2half_rn(v[i]);
                    else
                        static_cast<__nv_bfloat16 *>(y)[at] = __float2bfloat16_rn(v[i]);
                }
            }
            __syncwarp();
        }
        mm_fence_before();
    }
    if (S > 1) {
        cluster_sync_all();
        const int lo = 4 * (32 * rank / S), rows4 = (4 * (32 * (rank + 1) / S) - lo) / 4;
        for (int i = threadIdx.x; i < rows4 * toks; i += kMmThreads) {
            const int r = lo + 4 * (i % rows4), t = i / rows4;
            const uint32_t at = smem_addr(part + t * kMmRows + r);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s = 0; s < S; ++s) {
                const float4 v = ld_cluster_v4(map_to_rank(at, (uint32_t)s));
                acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
            }
            if (row0 + r < N) store_y4(y, type, (size_t)(tok0 + t) * N + row0 + r, N - row0 - r, acc);
        }
        cluster_sync_all();  // no CTA leaves while another reads its sums
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        mm_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols) : "memory");
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
    const int S = mx_split(row_tiles, tok_tiles, stages, c.num_sms);
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

template <bool kX8>
cudaError_t launch_mm_tokens(const LaunchCtx &c, MxType type, const MxMatmulArgs &a) {
    if (a.T <= 16) return launch_split<kX8, 16>(c, type, a);
    if (a.T <= 64) return launch_split<kX8, 64>(c, type, a);
    return launch_split<kX8, 128>(c, type, a);
}

}  // namespace

cudaError_t launch_mx_matmul(const LaunchCtx &c, MxType type, const MxMatmulArgs &a) {
    return a.x_bits == 8 ? launch_mm_tokens<true>(c, type, a) : launch_mm_tokens<false>(c, type, a);
}

}  // namespace q4mm

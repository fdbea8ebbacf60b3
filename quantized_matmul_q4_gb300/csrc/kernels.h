// Internal launchers behind the C ABI.  Each returns cudaSuccess or the
// launch error; arguments are already validated by capi.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <utility>

#include "attention_geometry.h"

namespace q4mm {

struct LaunchCtx {
    cudaStream_t stream;
    int num_sms;
    int max_smem_optin;  // bytes of shared memory a CTA may opt into
    int *status;         // device status word (bounded-wait time-outs)
    bool pdl;            // launch with programmatic stream serialization
    long long wait_limit;  // SM cycles a bounded in-kernel wait lasts at most
    int withhold;          // test only: a weight stage never copied (-1: none)
};

// Tensor memory.  An allocation that finds too few of an SM's 512 columns free
// waits until another CTA gives its own back, and the scheduler counts no
// columns: CTAs share an SM wherever threads, registers and shared memory
// allow.  So that no kernel of this library ever waits there for another (of
// two clusters, each could hold the SM that the other needs), shared memory
// keeps apart what does not fit: a kernel that allocates up to half of the
// columns takes at least kHalfTmemShared of it, so at most two such CTAs share
// an SM, and one that allocates more leaves less than kHalfTmemShared free.
// (Sizes with the 1 KB that the system adds to each CTA; asserted where the
// kernels' layouts are.)
constexpr uint32_t kSmShared = 228 * 1024;
constexpr uint32_t kCtaSharedExtra = 1024;
constexpr uint32_t kHalfTmemShared = 96 * 1024;
static_assert(3 * kHalfTmemShared > kSmShared, "two CTAs with half of the columns at most");

// Q4_K decode GEMV, 1..8 tokens on the one-token kernel (bulk-copied weight
// rows, byte planes of x in registers; each compute warp serves one token).
// Returns cudaErrorNotSupported when the shape is outside its geometry.
cudaError_t launch_q4k_gemv_t1(const LaunchCtx &c, const float *x, const uint8_t *W, float *y,
                               int K, int N, int T = 1);

// Q4_0 decode GEMV, one token (same kernel as the Q4_K one with the Q4_0
// row format).  cudaErrorNotSupported when the shape is outside its geometry.
cudaError_t launch_q4_0_gemv_t1(const LaunchCtx &c, const float *x, const uint8_t *W, float *y,
                                int K, int N, int T = 1);

// Q6_K decode GEMV, one token (the one-token kernel with the Q6_K row format).
cudaError_t launch_q6k_gemv_t1(const LaunchCtx &c, const float *x, const uint8_t *W, float *y, int K, int N,
                              int T = 1);

// BitNet b1.58 ternary GEMV, 1..8 tokens, on the same one-token kernel with
// the byte-plane integer code-dot (K % 256 == 0, W 16-byte aligned; otherwise
// cudaErrorNotSupported).
cudaError_t launch_ternary_gemv_t1(const LaunchCtx &c, const float *x, const uint8_t *W, float scale, float *y,
                                   int K, int N, int T = 1);

// Llama FFN input side, one token: h = silu(x·Wgᵀ)·(x·Wuᵀ), both Q4_K, in one
// launch of the one-token kernel (x split once for both weights).
cudaError_t launch_q4k_ffn_swiglu_t1(const LaunchCtx &c, const float *x, const uint8_t *Wg, const uint8_t *Wu,
                                     float *h, int K, int N);

// Q4_K decode GEMV for 1..8 tokens with x staged in shared memory.
cudaError_t launch_q4k_gemv_multi(const LaunchCtx &c, const float *x, const uint8_t *W, float *y,
                                  int K, int N, int T);
// The fused gate+up SwiGLU (h = silu(x·Wgᵀ) ⊙ (x·Wuᵀ)) for up to 8 tokens on
// the same kernel: one pass over both weights for all tokens.
cudaError_t launch_q4k_ffn_swiglu_multi(const LaunchCtx &c, const float *x, const uint8_t *Wg, const uint8_t *Wu,
                                        float *h, int K, int N, int T);

// Q4_K prefill, FP32 FMA (any token count, tiles of 64 tokens).
cudaError_t launch_q4k_mm_fp32(const LaunchCtx &c, const float *x, const uint8_t *W, float *y,
                               int K, int N, int T);

// Q4_K prefill on tcgen05 tensor cores (bf16 operands, fp32 accumulate).
cudaError_t launch_q4k_mm_tc(const LaunchCtx &c, const float *x, const uint8_t *W, float *y, int K,
                             int N, int T);

// The tensor-core prefill on a weight in the relayouted tensor-core layout
// (48 bytes per row and 64-value chunk), and the one-time relayout that
// makes it from a canonical Q4_K weight (q4k_relayout_tc_bytes(K, N) bytes).
cudaError_t launch_q4k_mm_tc_relayouted(const LaunchCtx &c, const float *x, const uint8_t *R, float *y, int K,
                                        int N, int T);
size_t q4k_relayout_tc_bytes(int K, int N);
cudaError_t launch_q4k_relayout_tc(const LaunchCtx &c, const uint8_t *W, uint8_t *R, int K, int N);

// The tensor-core prefill with its scratch in a fixed array of library
// memory (no allocation): bytes of scratch a call needs, and the launcher
// (cudaErrorInvalidValue if the need exceeds the array).
size_t q4k_mm_tc_scratch_bytes(int K, int N, int T);
cudaError_t launch_q4k_mm_tc_fixed_scratch(const LaunchCtx &c, const float *x, const uint8_t *W, float *y,
                                           int K, int N, int T);

// BitNet b1.58 ternary GEMV, any token count.
cudaError_t launch_ternary_gemv(const LaunchCtx &c, const float *x, const uint8_t *W, float scale,
                                float *y, int K, int N, int T);

// Microscaled (MX) operators; layouts in mx.cuh, contracts in q4mm.h.
enum class MxType { kF32 = 0, kF16 = 1, kBF16 = 2 };

// Quantises x [rows][K] (row stride in elements), or silu(x)·up where up is
// given, to `bits`-bit codes.
struct MxQuantizeArgs {
    const void *x;
    long long x_stride;
    const void *up;  // may be NULL
    long long up_stride;
    uint8_t *codes, *scales;
    int K, rows, bits;
};
cudaError_t launch_mx_quantize(const LaunchCtx &c, MxType type, const MxQuantizeArgs &a);

// h = x + residual, then h·(mean h² + eps)^-1/2·weight quantised; h is
// written where it is not NULL (it may be x or residual).
struct MxRmsnormArgs {
    const void *x;
    long long x_stride;
    const void *residual;  // may be NULL
    long long residual_stride;
    void *h;  // may be NULL
    long long h_stride;
    const void *weight;
    bool weight_f32;  // else x's type
    float eps;
    uint8_t *codes, *scales;
    int K, rows, bits;
};
cudaError_t launch_mx_rmsnorm(const LaunchCtx &c, MxType type, const MxRmsnormArgs &a);

struct MxDequantizeArgs {
    const uint8_t *codes, *scales;
    void *y;
    long long y_stride;
    int K, rows, bits;
};
cudaError_t launch_mx_dequantize(const LaunchCtx &c, MxType type, const MxDequantizeArgs &a);

// y[T][N] = x·wᵀ on the tensor cores, x in x_bits (4 or 8), w in 4 bits.
struct MxMatmulArgs {
    const uint8_t *x_codes, *x_scales, *w_codes, *w_scales;
    void *y;
    int K, N, T, x_bits;
};
cudaError_t launch_mx_matmul(const LaunchCtx &c, MxType type, const MxMatmulArgs &a);

// Bits of the device status word.
constexpr int kStatusTimeout = 1;  // a bounded wait ran out
constexpr int kStatusIndex = 2;    // a page number or position outside the cache or its table

// The paged MX cache and a batch of sequences in it; layouts in mx_cache.cuh.
struct MxCacheView {
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    int pages, heads, page, D, bits;
};
struct MxBatchView {
    const int *starts, *lengths, *table;
    int seqs, width;
};

// Rotation of a head's first `rotated` values (0: none).
struct RopeView {
    const double *frequencies;  // rotated / 2, radians per position
    int rotated;
    bool interleaved;  // pairs (2i, 2i + 1), else (i, i + rotated / 2)
    float magnitude;
};

struct RopeArgs {
    const void *x;
    long long x_token, x_head;
    const void *positions;
    bool positions_64;
    RopeView rope;
    void *out;  // may be x
    long long out_token, out_head;
    int tokens, heads, D;
};
cudaError_t launch_rope_rotate(const LaunchCtx &c, MxType type, const RopeArgs &a);

// k and v of the batch's rows, written to the cache or read from it.
struct MxCacheIoArgs {
    MxCacheView cache;
    MxBatchView batch;
    const void *k, *v;
    long long k_token, k_head, v_token, v_head;
    int tokens;
    int *status;
};
cudaError_t launch_mx_cache_write(const LaunchCtx &c, MxType type, const MxCacheIoArgs &a, const RopeView &rope);
cudaError_t launch_mx_cache_read(const LaunchCtx &c, MxType type, const MxCacheIoArgs &a);

// Attention of the batch's rows over the cache.
struct MxAttentionArgs {
    MxCacheView cache;
    MxBatchView batch;
    const void *q;
    long long q_token, q_head;
    void *y;
    long long y_token, y_head;
    float scale;
    bool causal;
    int tokens, heads;
    MxType type;
    bool vec;  // every four neighbouring values of q and y are aligned
    float *workspace;
    size_t workspace_bytes;
    int *status;
};
// Bytes of workspace that a split of few rows takes.
size_t mx_attention_few_workspace(int tokens, int heads, int kv_heads, int D, int seqs, const FewSplit &f);
// few rows a kv head; tiles of 128, on tcgen05 (as_f32: whatever the type)
cudaError_t launch_mx_attention_few(const LaunchCtx &c, const MxAttentionArgs &a, const FewSplit &f, bool as_f32);
cudaError_t launch_mx_attention_many(const LaunchCtx &c, const MxAttentionArgs &a, int split, bool as_f32);

// Raise a kernel's dynamic shared-memory limit to at least `bytes` on the
// current device; the attribute call is made only when the limit grows, so a
// warmed-up launch (for instance one being captured into a CUDA graph) issues
// nothing but the launch itself.
cudaError_t ensure_smem_limit(const void *kernel, size_t bytes);

template <typename... KArgs>
cudaError_t ensure_smem(void (*kernel)(KArgs...), size_t bytes) {
    return ensure_smem_limit(reinterpret_cast<const void *>(kernel), bytes);
}

// Launch helper: cudaLaunchKernelEx with optional programmatic serialization.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(const LaunchCtx &c, void (*kernel)(KArgs...), dim3 grid, dim3 block,
                          size_t smem, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];
    int nattr = 0;
    if (c.pdl) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        nattr = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = nattr;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace q4mm

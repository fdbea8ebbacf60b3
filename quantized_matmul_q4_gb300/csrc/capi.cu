// C ABI of libq4mm.so: argument validation, dispatch to the kernels, error
// reporting.  Declarations and the contract of every entry point are in
// include/q4mm.h.
#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "q4mm.h"
#include "attention_geometry.h"
#include "dispatch.h"
#include "kernels.h"
#include "sync.cuh"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return code;
}

int fail_cuda(cudaError_t e, const char *what) {
    return fail(Q4MM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Set by a kernel whose bounded wait gave up.
__device__ int g_device_status;

struct DeviceInfo {
    // Set (release) after the other fields are filled; read (acquire) without
    // the lock, so a thread that sees it set also sees those fields.
    std::atomic<bool> ready{false};
    int num_sms = 0;
    int max_smem_optin = 0;
    int *status = nullptr;
};

constexpr int kMaxDevices = 64;
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

// Armed by q4mm_test_fail_next_wait for the calling thread's next compute
// call only.
struct TestFault {
    bool armed = false;
    int stage = -1;
    long long limit = 0;
};
thread_local TestFault g_test_fault;

void take_fault(q4mm::LaunchCtx *ctx) {
    if (!g_test_fault.armed) return;
    ctx->wait_limit = g_test_fault.limit;
    ctx->withhold = g_test_fault.stage;
    g_test_fault.armed = false;
}

// The kernel that the calling thread's attention calls take, set by
// q4mm_test_attention_kernel: 0 as planned, 1 few rows, 2 many.
thread_local int g_test_attention = 0;

int attention_chain(int dtype) {
    return dtype == Q4MM_F16 ? q4mm::kChainF16 : dtype == Q4MM_BF16 ? q4mm::kChainBf16 : 0;
}

q4mm::AttentionPlan plan_attention(int tokens, int heads, int kv_heads, int seqs, int width, int page, int dtype,
                                   int num_sms) {
    const int chain = attention_chain(dtype);
    q4mm::AttentionPlan p = q4mm::attention_plan(tokens, heads / kv_heads, seqs, kv_heads, q4mm::table_keys(width, page),
                                                 dtype == Q4MM_F32, num_sms, chain);
    if (g_test_attention) p.many = g_test_attention == 2;
    return p;
}

// take_test_fault: a compute call (it consumes an armed test fault).
int device_ctx(q4mm_stream_t stream, q4mm::LaunchCtx *ctx, bool take_test_fault = true) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(Q4MM_ERR_CUDA, "device ordinal %d out of range", dev);
    DeviceInfo &d = g_dev[dev];
    if (!d.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_dev_mu);
        if (!d.ready.load(std::memory_order_relaxed)) {
            e = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
            if (e != cudaSuccess) return fail_cuda(e, "cudaDeviceGetAttribute(SM count)");
            e = cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
            if (e != cudaSuccess) return fail_cuda(e, "cudaDeviceGetAttribute(shared memory)");
            e = cudaGetSymbolAddress(reinterpret_cast<void **>(&d.status), g_device_status);
            if (e != cudaSuccess) return fail_cuda(e, "cudaGetSymbolAddress(status)");
            d.ready.store(true, std::memory_order_release);
        }
    }
    ctx->stream = reinterpret_cast<cudaStream_t>(stream);
    ctx->num_sms = d.num_sms;
    ctx->max_smem_optin = d.max_smem_optin;
    ctx->status = d.status;
    // Programmatic dependent launch: a kernel may start its weight stream
    // while the previous kernel on the stream finishes.
    ctx->pdl = true;
    ctx->wait_limit = q4mm::kWaitLimitCycles;
    ctx->withhold = -1;
    if (take_test_fault) take_fault(ctx);
    return Q4MM_OK;
}

// Runs a one-token-kernel launcher over the tokens in chunks of up to 8,
// halving a chunk whose geometry the kernel cannot hold.
template <class F>
cudaError_t token_chunks(F launch, const float *x, float *y, int K, int N, int tokens) {
    cudaError_t e = cudaSuccess;
    for (int t0 = 0; t0 < tokens && e == cudaSuccess;) {
        int tt = tokens - t0 < 8 ? tokens - t0 : 8;
        for (;;) {
            e = launch(x + (size_t)t0 * K, y + (size_t)t0 * N, tt);
            if (e != cudaErrorNotSupported || tt == 1) break;
            tt /= 2;
        }
        t0 += tt;
    }
    return e;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

// w_bytes_per_row: the weight's bytes per output row; w_total_bytes, when
// nonzero, its whole size instead (a layout padded past N rows).
int check_common(const float *x, const void *w, const float *y, int K, int N, int T, int k_multiple,
                 size_t w_bytes_per_row, size_t w_align, size_t w_total_bytes = 0) {
    if (!x || !w || !y) return fail(Q4MM_ERR_NULL, "x, weight and y must be non-NULL");
    if (K <= 0 || N <= 0 || T <= 0)
        return fail(Q4MM_ERR_DIM, "inputDim (%d), outputDim (%d) and tokens (%d) must be positive", K, N, T);
    if (K % k_multiple)
        return fail(Q4MM_ERR_DIM, "inputDim %d is not a multiple of %d", K, k_multiple);
    if (K > Q4MM_MAX_INPUT_DIM)
        return fail(Q4MM_ERR_DIM, "inputDim %d exceeds the limit %d", K, Q4MM_MAX_INPUT_DIM);
    if (reinterpret_cast<uintptr_t>(x) % 16) return fail(Q4MM_ERR_ALIGN, "x must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(y) % 4) return fail(Q4MM_ERR_ALIGN, "y must be 4-byte aligned");
    if (reinterpret_cast<uintptr_t>(w) % w_align)
        return fail(Q4MM_ERR_ALIGN, "weight must be %zu-byte aligned", w_align);
    const size_t xb = (size_t)T * K * sizeof(float), yb = (size_t)T * N * sizeof(float);
    const size_t wb = w_total_bytes ? w_total_bytes : (size_t)N * w_bytes_per_row;
    if (overlap(x, xb, y, yb) || overlap(x, xb, w, wb) || overlap(w, wb, y, yb))
        return fail(Q4MM_ERR_ALIAS, "x, weight and y must not overlap");
    return Q4MM_OK;
}

// Checks shared by the MX entry points.

size_t mx_size(int dtype) { return dtype == Q4MM_F32 ? 4 : 2; }

int check_mx_dims(int K, int rows, int bits, const char *rows_name) {
    if (K <= 0 || rows < 0)
        return fail(Q4MM_ERR_DIM, "inputDim (%d) must be positive and %s (%d) not negative", K, rows_name, rows);
    if (K > Q4MM_MAX_INPUT_DIM) return fail(Q4MM_ERR_DIM, "inputDim %d exceeds the limit %d", K, Q4MM_MAX_INPUT_DIM);
    if (rows > Q4MM_MX_MAX_ROWS)
        return fail(Q4MM_ERR_DIM, "%s (%d) exceeds the limit %d", rows_name, rows, Q4MM_MX_MAX_ROWS);
    if (bits != 4 && bits != 8) return fail(Q4MM_ERR_DIM, "bits (%d) must be 4 or 8", bits);
    return Q4MM_OK;
}

int check_mx_dtype(int dtype, const char *what) {
    if (dtype != Q4MM_F32 && dtype != Q4MM_F16 && dtype != Q4MM_BF16)
        return fail(Q4MM_ERR_DIM, "%s type (%d) must be Q4MM_F32, Q4MM_F16 or Q4MM_BF16", what, dtype);
    return Q4MM_OK;
}

// One buffer of a call: [p, p + bytes).
struct Span {
    const void *p;
    size_t bytes;
    const char *name;
};

// The bytes that `rows` strided rows of K values reach over.
Span mx_rows(const void *p, long long stride, int K, int rows, size_t size, const char *name) {
    return Span{p, ((size_t)(rows - 1) * (size_t)stride + (size_t)K) * size, name};
}
Span mx_codes(const void *p, int K, int rows, int bits, const char *name) {
    return Span{p, Q4MM_MX_CODE_BYTES(K, rows, bits), name};
}
Span mx_scales(const void *p, int K, int rows, const char *name) {
    return Span{p, Q4MM_MX_SCALE_BYTES(K, rows), name};
}

// Strides count elements; one row has none.  Rows that reach past 2^48
// elements are no memory's (and would overflow the sums below).
int check_mx_stride(long long stride, int K, int rows, const char *name) {
    if (rows == 1) return Q4MM_OK;
    if (stride < K) return fail(Q4MM_ERR_DIM, "the row stride of %s (%lld) is below its row of %d", name, stride, K);
    if (stride > (1LL << 48) / (rows - 1))
        return fail(Q4MM_ERR_DIM, "%d rows of %s %lld elements apart do not fit in memory", rows, name, stride);
    return Q4MM_OK;
}

int check_mx_ptr(const Span &s, size_t align) {
    if (!s.p) return fail(Q4MM_ERR_NULL, "%s must be non-NULL", s.name);
    if (reinterpret_cast<uintptr_t>(s.p) % align)
        return fail(Q4MM_ERR_ALIGN, "%s must be %zu-byte aligned", s.name, align);
    return Q4MM_OK;
}

// No output may overlap an input or another output.
int check_mx_alias(const Span *outs, int nouts, const Span *ins, int nins) {
    for (int i = 0; i < nouts; ++i) {
        for (int j = i + 1; j < nouts; ++j)
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
                return fail(Q4MM_ERR_ALIAS, "%s and %s must not overlap", outs[i].name, outs[j].name);
        for (int j = 0; j < nins; ++j)
            if (ins[j].p && overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes))
                return fail(Q4MM_ERR_ALIAS, "%s and %s must not overlap", outs[i].name, ins[j].name);
    }
    return Q4MM_OK;
}

// Checks shared by the entry points of attention.

// The bytes that [tokens][heads][D] values with these strides reach over
// (strides are checked first).
Span head_span(const void *p, long long token, long long head, int tokens, int heads, int D, size_t size,
               const char *name) {
    return Span{p, ((size_t)(tokens - 1) * (size_t)token + (size_t)(heads - 1) * (size_t)head + (size_t)D) * size, name};
}

// A token's heads, or a head's tokens, may lie inside each other's gaps, but
// not on each other (`writes`); strides are not negative.
int check_head_strides(long long token, long long head, int tokens, int heads, int D, bool writes, const char *name) {
    if ((tokens > 1 && token < 0) || (heads > 1 && head < 0))
        return fail(Q4MM_ERR_DIM, "the strides of %s (%lld, %lld) must not be negative", name, token, head);
    if ((tokens > 1 && token > (1LL << 46) / (tokens - 1)) || (heads > 1 && head > (1LL << 46) / (heads - 1)))
        return fail(Q4MM_ERR_DIM, "%s does not fit in memory with strides %lld and %lld", name, token, head);
    if (writes) {
        const bool tokens_outside =
            (heads == 1 || head >= D) && (tokens == 1 || token >= (heads - 1) * (heads > 1 ? head : 0) + D);
        const bool heads_outside =
            (tokens == 1 || token >= D) && (heads == 1 || head >= (tokens - 1) * (tokens > 1 ? token : 0) + D);
        if (!tokens_outside && !heads_outside)
            return fail(Q4MM_ERR_ALIAS, "the heads of %s overlap with strides %lld and %lld", name, token, head);
    }
    return Q4MM_OK;
}

int check_rope(const double *frequencies, int rotated, float magnitude, int D) {
    if (rotated < 0 || rotated > D || rotated % 2)
        return fail(Q4MM_ERR_DIM, "rotated (%d) must be even and between 0 and headDim (%d)", rotated, D);
    if (!(magnitude - magnitude == 0.f)) return fail(Q4MM_ERR_DIM, "magnitude must be finite");
    if (rotated == 0) return Q4MM_OK;
    return check_mx_ptr(Span{frequencies, (size_t)rotated / 2 * 8, "frequencies"}, 8);
}

// The rows that share a key head are numbered in 32 bits (a tile's last ones may not exist).
int check_rows(int tokens, int group) {
    if ((long long)tokens * group <= Q4MM_MX_MAX_ROWS) return Q4MM_OK;
    return fail(Q4MM_ERR_DIM, "tokens (%d) times heads of a key head (%d) must be at most %d rows", tokens, group,
                Q4MM_MX_MAX_ROWS);
}

struct CacheCall {
    q4mm::MxCacheView cache;
    q4mm::MxBatchView batch;
    Span spans[7];  // codes and scales of k and v, then starts, lengths, table
};

// Sizes and pointers of a cache and a batch.
int check_cache(CacheCall &c, int tokens) {
    const q4mm::MxCacheView &m = c.cache;
    const q4mm::MxBatchView &b = c.batch;
    if (m.D != 32 && m.D != 64 && m.D != 96 && m.D != 128)
        return fail(Q4MM_ERR_DIM, "headDim (%d) must be 32, 64, 96 or 128", m.D);
    if (m.bits != 4 && m.bits != 8) return fail(Q4MM_ERR_DIM, "bits (%d) must be 4 or 8", m.bits);
    if (m.pages <= 0 || m.heads <= 0 || m.heads > Q4MM_MX_MAX_HEADS)
        return fail(Q4MM_ERR_DIM, "pages (%d) and kvHeads (%d, at most %d) must be positive", m.pages, m.heads,
                    Q4MM_MX_MAX_HEADS);
    if (m.page <= 0 || m.page % 16 || m.page > (1 << 24))
        return fail(Q4MM_ERR_DIM, "pageTokens (%d) must be a positive multiple of 16, at most 2^24", m.page);
    if (b.seqs < 0 || b.seqs > (1 << 24) || b.width < 0)
        return fail(Q4MM_ERR_DIM, "sequences (%d, at most 2^24) and tableWidth (%d) must not be negative", b.seqs,
                    b.width);
    if (tokens < 0 || tokens > Q4MM_MX_MAX_ROWS)
        return fail(Q4MM_ERR_DIM, "tokens (%d) must be between 0 and %d", tokens, Q4MM_MX_MAX_ROWS);
    const size_t slots = (size_t)m.pages * m.heads * m.page;
    const size_t codes = slots * (m.D * m.bits / 8);
    c.spans[0] = Span{m.k_codes, codes, "k_codes"}, c.spans[1] = Span{m.k_scales, slots * 4, "k_scales"};
    c.spans[2] = Span{m.v_codes, codes, "v_codes"}, c.spans[3] = Span{m.v_scales, slots * 4, "v_scales"};
    c.spans[4] = Span{b.starts, ((size_t)b.seqs + 1) * 4, "starts"}, c.spans[5] = Span{b.lengths, (size_t)b.seqs * 4, "lengths"};
    c.spans[6] = Span{b.table, (size_t)b.seqs * b.width * 4, "table"};
    int rc;
    for (int i = 0; i < 7; ++i) {
        if (b.seqs == 0 && i >= 4) break;
        if (b.width == 0 && i == 6) break;
        if ((rc = check_mx_ptr(c.spans[i], i < 4 ? 16 : 4))) return rc;
    }
    return Q4MM_OK;
}

int mx_quantize_call(const void *x, long long x_stride, const void *up, long long up_stride, bool swiglu, int dtype,
                     void *codes, void *scales, int K, int rows, int bits, q4mm_stream_t stream) {
    int rc = check_mx_dims(K, rows, bits, "rows");
    if (rc || (rc = check_mx_dtype(dtype, "input"))) return rc;
    if (rows == 0) return Q4MM_OK;
    const size_t size = mx_size(dtype);
    const char *xn = swiglu ? "gate" : "x";
    if ((rc = check_mx_stride(x_stride, K, rows, xn)) ||
        (swiglu && (rc = check_mx_stride(up_stride, K, rows, "up"))))
        return rc;
    const Span ins[2] = {mx_rows(x, x_stride, K, rows, size, xn), mx_rows(up, up_stride, K, rows, size, "up")};
    const Span outs[2] = {mx_codes(codes, K, rows, bits, "codes"), mx_scales(scales, K, rows, "scales")};
    if ((rc = check_mx_ptr(ins[0], size)) || (swiglu && (rc = check_mx_ptr(ins[1], size))) ||
        (rc = check_mx_ptr(outs[0], 32)) || (rc = check_mx_ptr(outs[1], 16)) ||
        (rc = check_mx_alias(outs, 2, ins, swiglu ? 2 : 1)))
        return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx, false))) return rc;
    const q4mm::MxQuantizeArgs a{x, x_stride, swiglu ? up : nullptr, up_stride, static_cast<uint8_t *>(codes),
                                 static_cast<uint8_t *>(scales), K, rows, bits};
    const cudaError_t e = q4mm::launch_mx_quantize(ctx, static_cast<q4mm::MxType>(dtype), a);
    if (e != cudaSuccess) return fail_cuda(e, swiglu ? "mx_swiglu launch" : "mx_quantize launch");
    return Q4MM_OK;
}

}  // namespace

namespace q4mm {

cudaError_t ensure_smem_limit(const void *kernel, size_t bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    struct Entry {
        int dev;
        const void *fn;
        size_t bytes;
    };
    static Entry table[256];
    static int used = 0;
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (table[i].dev == dev && table[i].fn == kernel && table[i].bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    // The largest shared-memory configuration of the SM: kernels that pair a
    // CTA of the next launch with one of the current launch need both to fit.
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < used; ++i)
        if (table[i].dev == dev && table[i].fn == kernel) {
            table[i].bytes = bytes;
            return cudaSuccess;
        }
    if (used < 256) table[used++] = Entry{dev, kernel, bytes};
    return cudaSuccess;
}

}  // namespace q4mm

extern "C" {

int q4k_matmul(const float *x, const void *w_q4k, float *y, int inputDim, int outputDim, int tokens,
               q4mm_stream_t stream) {
    int rc = check_common(x, w_q4k, y, inputDim, outputDim, tokens, 256,
                          (size_t)(inputDim / 256) * 144, 16);
    if (rc) return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    const uint8_t *W = static_cast<const uint8_t *>(w_q4k);
    // The kernel for this token count (dispatch.h), each falling back to the
    // next where its geometry does not fit the shape.
    const q4mm::Q4kPath path = q4mm::q4k_matmul_path(tokens, outputDim, ctx.num_sms);
    cudaError_t e = cudaErrorNotSupported;
    if (path == q4mm::Q4kPath::kOneToken) e = q4mm::launch_q4k_gemv_t1(ctx, x, W, y, inputDim, outputDim, tokens);
    if (e == cudaErrorNotSupported && tokens <= 8)
        e = q4mm::launch_q4k_gemv_multi(ctx, x, W, y, inputDim, outputDim, tokens);
    if (e == cudaErrorNotSupported && path == q4mm::Q4kPath::kTileChunks) {
        e = cudaSuccess;
        for (int t0 = 0; t0 < tokens && e == cudaSuccess; t0 += 8) {
            const int tt = tokens - t0 < 8 ? tokens - t0 : 8;
            e = q4mm::launch_q4k_gemv_multi(ctx, x + (size_t)t0 * inputDim, W, y + (size_t)t0 * outputDim, inputDim,
                                            outputDim, tt);
            // A geometry the register-tile kernel cannot hold fails on the
            // first chunk, before anything is launched.
            if (e == cudaErrorNotSupported && t0 > 0) return fail_cuda(e, "q4k_matmul launch");
        }
    }
    if (e == cudaErrorNotSupported) e = q4mm::launch_q4k_mm_fp32(ctx, x, W, y, inputDim, outputDim, tokens);
    if (e != cudaSuccess) return fail_cuda(e, "q4k_matmul launch");
    return Q4MM_OK;
}

int q4k_matmul_tc(const float *x, const void *w_q4k, float *y, int inputDim, int outputDim,
                  int tokens, q4mm_stream_t stream) {
    int rc = check_common(x, w_q4k, y, inputDim, outputDim, tokens, 256,
                          (size_t)(inputDim / 256) * 144, 16);
    if (rc) return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    cudaError_t e = q4mm::launch_q4k_mm_tc(ctx, x, static_cast<const uint8_t *>(w_q4k), y, inputDim,
                                           outputDim, tokens);
    if (e != cudaSuccess) return fail_cuda(e, "q4k_matmul_tc launch");
    return Q4MM_OK;
}

int q4k_matmul_tc_noalloc(const float *x, const void *w_q4k, float *y, int inputDim, int outputDim,
                          int tokens, q4mm_stream_t stream) {
    int rc = check_common(x, w_q4k, y, inputDim, outputDim, tokens, 256,
                          (size_t)(inputDim / 256) * 144, 16);
    if (rc) return rc;
    const size_t need = q4mm::q4k_mm_tc_scratch_bytes(inputDim, outputDim, tokens);
    if (need > (size_t)Q4MM_TC_NOALLOC_SCRATCH_BYTES)
        return fail(Q4MM_ERR_DIM,
                    "q4k_matmul_tc_noalloc: %d tokens x inputDim %d x outputDim %d need %zu bytes of scratch, "
                    "more than the fixed %zu-byte array (use q4k_matmul_tc, or fewer tokens per call)",
                    tokens, inputDim, outputDim, need, (size_t)Q4MM_TC_NOALLOC_SCRATCH_BYTES);
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    cudaError_t e = q4mm::launch_q4k_mm_tc_fixed_scratch(ctx, x, static_cast<const uint8_t *>(w_q4k), y,
                                                         inputDim, outputDim, tokens);
    if (e != cudaSuccess) return fail_cuda(e, "q4k_matmul_tc_noalloc launch");
    return Q4MM_OK;
}

int q4k_relayout_tc(const void *w_q4k, void *w_tc, int inputDim, int outputDim, q4mm_stream_t stream) {
    if (!w_q4k || !w_tc) return fail(Q4MM_ERR_NULL, "w_q4k and w_tc must be non-NULL");
    if (inputDim <= 0 || outputDim <= 0)
        return fail(Q4MM_ERR_DIM, "inputDim (%d) and outputDim (%d) must be positive", inputDim, outputDim);
    if (inputDim % 256) return fail(Q4MM_ERR_DIM, "inputDim %d is not a multiple of 256", inputDim);
    if (inputDim > Q4MM_MAX_INPUT_DIM)
        return fail(Q4MM_ERR_DIM, "inputDim %d exceeds the limit %d", inputDim, Q4MM_MAX_INPUT_DIM);
    if (reinterpret_cast<uintptr_t>(w_q4k) % 16 || reinterpret_cast<uintptr_t>(w_tc) % 16)
        return fail(Q4MM_ERR_ALIGN, "w_q4k and w_tc must be 16-byte aligned");
    const size_t wb = (size_t)outputDim * (inputDim / 256) * 144;
    if (overlap(w_q4k, wb, w_tc, Q4MM_TC_RELAYOUT_BYTES(inputDim, outputDim)))
        return fail(Q4MM_ERR_ALIAS, "w_q4k and w_tc must not overlap");
    q4mm::LaunchCtx ctx;
    int rc;
    if ((rc = device_ctx(stream, &ctx, false))) return rc;
    const cudaError_t e = q4mm::launch_q4k_relayout_tc(ctx, static_cast<const uint8_t *>(w_q4k),
                                                       static_cast<uint8_t *>(w_tc), inputDim, outputDim);
    if (e != cudaSuccess) return fail_cuda(e, "q4k_relayout_tc launch");
    return Q4MM_OK;
}

int q4k_matmul_tc_relayouted(const float *x, const void *w_tc, float *y, int inputDim, int outputDim, int tokens,
                             q4mm_stream_t stream) {
    // The weight-overlap check takes the padded layout's exact size.
    int rc = check_common(x, w_tc, y, inputDim, outputDim, tokens, 256, 0, 16,
                          inputDim > 0 && outputDim > 0 ? Q4MM_TC_RELAYOUT_BYTES(inputDim, outputDim) : 0);
    if (rc) return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    cudaError_t e = q4mm::launch_q4k_mm_tc_relayouted(ctx, x, static_cast<const uint8_t *>(w_tc), y, inputDim,
                                                      outputDim, tokens);
    if (e != cudaSuccess) return fail_cuda(e, "q4k_matmul_tc_relayouted launch");
    return Q4MM_OK;
}

int q4_0_gemv(const float *x, const void *w_q4_0, float *y, int inputDim, int outputDim, int tokens,
              q4mm_stream_t stream) {
    int rc = check_common(x, w_q4_0, y, inputDim, outputDim, tokens, 256,
                          (size_t)(inputDim / 32) * 18, 16);
    if (rc) return rc;
    if (inputDim > Q4MM_Q4_0_MAX_INPUT_DIM)
        return fail(Q4MM_ERR_DIM, "inputDim %d exceeds the Q4_0 limit %d", inputDim, Q4MM_Q4_0_MAX_INPUT_DIM);
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    const uint8_t *W = static_cast<const uint8_t *>(w_q4_0);
    const cudaError_t e = token_chunks(
        [&](const float *xt, float *yt, int tt) {
            return q4mm::launch_q4_0_gemv_t1(ctx, xt, W, yt, inputDim, outputDim, tt);
        },
        x, y, inputDim, outputDim, tokens);
    if (e != cudaSuccess) return fail_cuda(e, "q4_0_gemv launch");
    return Q4MM_OK;
}

int q6k_gemv(const float *x, const void *w_q6k, float *y, int inputDim, int outputDim, int tokens,
             q4mm_stream_t stream) {
    int rc = check_common(x, w_q6k, y, inputDim, outputDim, tokens, 256, (size_t)(inputDim / 256) * 210, 16);
    if (rc) return rc;
    if (inputDim > Q4MM_Q6K_MAX_INPUT_DIM)
        return fail(Q4MM_ERR_DIM, "inputDim %d exceeds the Q6_K limit %d", inputDim, Q4MM_Q6K_MAX_INPUT_DIM);
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    const uint8_t *W = static_cast<const uint8_t *>(w_q6k);
    const cudaError_t e = token_chunks(
        [&](const float *xt, float *yt, int tt) {
            return q4mm::launch_q6k_gemv_t1(ctx, xt, W, yt, inputDim, outputDim, tt);
        },
        x, y, inputDim, outputDim, tokens);
    if (e != cudaSuccess) return fail_cuda(e, "q6k_gemv launch");
    return Q4MM_OK;
}

int q4k_ffn_swiglu(const float *x, const void *w_gate, const void *w_up, float *h, int inputDim,
                   int hiddenDim, int tokens, q4mm_stream_t stream) {
    const size_t row_bytes = (size_t)(inputDim / 256) * 144;
    int rc = check_common(x, w_gate, h, inputDim, hiddenDim, tokens, 256, row_bytes, 16);
    if (rc) return rc;
    if ((rc = check_common(x, w_up, h, inputDim, hiddenDim, tokens, 256, row_bytes, 16))) return rc;
    if (inputDim > Q4MM_FFN_MAX_INPUT_DIM)
        return fail(Q4MM_ERR_DIM, "inputDim %d exceeds the fused FFN limit %d", inputDim, Q4MM_FFN_MAX_INPUT_DIM);
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    const uint8_t *Wg = static_cast<const uint8_t *>(w_gate), *Wu = static_cast<const uint8_t *>(w_up);
    // From 3 tokens on: the FP32 register-tile kernel over both weights, up
    // to 8 tokens per pass; 1-2 tokens (or a geometry it cannot hold): the
    // one-token kernel, one launch per token.
    if (tokens >= 3) {
        cudaError_t e = cudaSuccess;
        for (int t0 = 0; t0 < tokens && e == cudaSuccess; t0 += 8) {
            const int tt = tokens - t0 < 8 ? tokens - t0 : 8;
            e = q4mm::launch_q4k_ffn_swiglu_multi(ctx, x + (size_t)t0 * inputDim, Wg, Wu, h + (size_t)t0 * hiddenDim,
                                                  inputDim, hiddenDim, tt);
            if (e == cudaErrorNotSupported && t0 == 0) break;  // nothing launched yet
        }
        if (e == cudaSuccess) return Q4MM_OK;
        if (e != cudaErrorNotSupported) return fail_cuda(e, "q4k_ffn_swiglu launch");
    }
    for (int t = 0; t < tokens; ++t) {
        const cudaError_t e = q4mm::launch_q4k_ffn_swiglu_t1(ctx, x + (size_t)t * inputDim, Wg, Wu,
                                                             h + (size_t)t * hiddenDim, inputDim, hiddenDim);
        if (e != cudaSuccess) return fail_cuda(e, "q4k_ffn_swiglu launch");
    }
    return Q4MM_OK;
}

int ternary_gemv(const float *x, const void *w_packed, float scale, float *y, int inputDim,
                 int outputDim, int tokens, q4mm_stream_t stream) {
    int rc = check_common(x, w_packed, y, inputDim, outputDim, tokens, 4, (size_t)inputDim / 4, 1);
    if (rc) return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    cudaError_t e = q4mm::launch_ternary_gemv(ctx, x, static_cast<const uint8_t *>(w_packed), scale, y,
                                              inputDim, outputDim, tokens);
    if (e != cudaSuccess) return fail_cuda(e, "ternary_gemv launch");
    return Q4MM_OK;
}

int mx_quantize(const void *x, long long x_stride, int dtype, void *codes, void *scales, int inputDim, int rows,
                int bits, q4mm_stream_t stream) {
    return mx_quantize_call(x, x_stride, nullptr, 0, false, dtype, codes, scales, inputDim, rows, bits, stream);
}

int mx_swiglu(const void *gate, long long gate_stride, const void *up, long long up_stride, int dtype, void *codes,
              void *scales, int hiddenDim, int rows, int bits, q4mm_stream_t stream) {
    return mx_quantize_call(gate, gate_stride, up, up_stride, true, dtype, codes, scales, hiddenDim, rows, bits,
                            stream);
}

int mx_rmsnorm(const void *x, long long x_stride, const void *residual, long long residual_stride, void *h,
               long long h_stride, int dtype, const void *weight, int weight_dtype, float eps, void *codes,
               void *scales, int inputDim, int rows, int bits, q4mm_stream_t stream) {
    const int K = inputDim;
    int rc = check_mx_dims(K, rows, bits, "rows");
    if (rc || (rc = check_mx_dtype(dtype, "input")) || (rc = check_mx_dtype(weight_dtype, "weight"))) return rc;
    if (weight_dtype != dtype && weight_dtype != Q4MM_F32)
        return fail(Q4MM_ERR_DIM, "the weight's type must be the input's or Q4MM_F32");
    if (!(eps >= 0.f)) return fail(Q4MM_ERR_DIM, "eps (%g) must not be negative", (double)eps);
    if (rows == 0) return Q4MM_OK;
    const size_t size = mx_size(dtype), wsize = mx_size(weight_dtype);
    if ((rc = check_mx_stride(x_stride, K, rows, "x")) ||
        (residual && (rc = check_mx_stride(residual_stride, K, rows, "residual"))) ||
        (h && (rc = check_mx_stride(h_stride, K, rows, "h"))))
        return rc;
    const Span xs = mx_rows(x, x_stride, K, rows, size, "x"), ws{weight, (size_t)K * wsize, "weight"};
    const Span rs = mx_rows(residual, residual_stride, K, rows, size, "residual");
    const Span hs = mx_rows(h, h_stride, K, rows, size, "h");
    const Span outs[3] = {mx_codes(codes, K, rows, bits, "codes"), mx_scales(scales, K, rows, "scales"), hs};
    if ((rc = check_mx_ptr(xs, size)) || (rc = check_mx_ptr(ws, wsize)) ||
        (residual && (rc = check_mx_ptr(rs, size))) || (h && (rc = check_mx_ptr(hs, size))) ||
        (rc = check_mx_ptr(outs[0], 32)) || (rc = check_mx_ptr(outs[1], 16)))
        return rc;
    const Span ins[3] = {xs, ws, rs};
    if ((rc = check_mx_alias(outs, h ? 3 : 2, ins, 0)) || (rc = check_mx_alias(outs, 2, ins, 3))) return rc;
    // h may be x or the residual itself (the same rows), not a part of them.
    const Span same[2] = {xs, rs};
    for (int i = 0; i < 2; ++i) {
        const bool itself = same[i].p == h && (rows == 1 || (i == 0 ? x_stride : residual_stride) == h_stride);
        if (h && same[i].p && !itself && (rc = check_mx_alias(&hs, 1, &same[i], 1))) return rc;
    }
    if (h && (rc = check_mx_alias(&hs, 1, &ws, 1))) return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx, false))) return rc;
    const q4mm::MxRmsnormArgs a{x, x_stride, residual, residual_stride, h, h_stride, weight,
                                weight_dtype == Q4MM_F32, eps, static_cast<uint8_t *>(codes),
                                static_cast<uint8_t *>(scales), K, rows, bits};
    const cudaError_t e = q4mm::launch_mx_rmsnorm(ctx, static_cast<q4mm::MxType>(dtype), a);
    if (e != cudaSuccess) return fail_cuda(e, "mx_rmsnorm launch");
    return Q4MM_OK;
}

int mx_dequantize(const void *codes, const void *scales, void *y, long long y_stride, int dtype, int inputDim,
                  int rows, int bits, q4mm_stream_t stream) {
    const int K = inputDim;
    int rc = check_mx_dims(K, rows, bits, "rows");
    if (rc || (rc = check_mx_dtype(dtype, "output"))) return rc;
    if (rows == 0) return Q4MM_OK;
    if ((rc = check_mx_stride(y_stride, K, rows, "y"))) return rc;
    const Span out = mx_rows(y, y_stride, K, rows, mx_size(dtype), "y");
    const Span ins[2] = {mx_codes(codes, K, rows, bits, "codes"), mx_scales(scales, K, rows, "scales")};
    if ((rc = check_mx_ptr(out, mx_size(dtype))) || (rc = check_mx_ptr(ins[0], 32)) ||
        (rc = check_mx_ptr(ins[1], 16)) || (rc = check_mx_alias(&out, 1, ins, 2)))
        return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx, false))) return rc;
    const q4mm::MxDequantizeArgs a{static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), y,
                                   y_stride, K, rows, bits};
    const cudaError_t e = q4mm::launch_mx_dequantize(ctx, static_cast<q4mm::MxType>(dtype), a);
    if (e != cudaSuccess) return fail_cuda(e, "mx_dequantize launch");
    return Q4MM_OK;
}

int mx_matmul(const void *x_codes, const void *x_scales, int x_bits, const void *w_codes, const void *w_scales,
              void *y, int dtype, int inputDim, int outputDim, int tokens, q4mm_stream_t stream) {
    const int K = inputDim, N = outputDim, T = tokens;
    int rc = check_mx_dims(K, T, x_bits, "tokens");
    if (rc || (rc = check_mx_dtype(dtype, "output"))) return rc;
    if (N <= 0 || N > Q4MM_MX_MAX_ROWS)
        return fail(Q4MM_ERR_DIM, "outputDim (%d) must be positive and at most %d", N, Q4MM_MX_MAX_ROWS);
    if (T == 0) return Q4MM_OK;
    const Span out{y, (size_t)T * N * mx_size(dtype), "y"};
    const Span ins[4] = {mx_codes(x_codes, K, T, x_bits, "x_codes"), mx_scales(x_scales, K, T, "x_scales"),
                         mx_codes(w_codes, K, N, 4, "w_codes"), mx_scales(w_scales, K, N, "w_scales")};
    for (int i = 0; i < 4; ++i)
        if ((rc = check_mx_ptr(ins[i], i % 2 ? 16 : 32))) return rc;
    if ((rc = check_mx_ptr(out, mx_size(dtype))) || (rc = check_mx_alias(&out, 1, ins, 4))) return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx))) return rc;
    const q4mm::MxMatmulArgs a{static_cast<const uint8_t *>(x_codes), static_cast<const uint8_t *>(x_scales),
                               static_cast<const uint8_t *>(w_codes), static_cast<const uint8_t *>(w_scales), y,
                               K, N, T, x_bits};
    const cudaError_t e = q4mm::launch_mx_matmul(ctx, static_cast<q4mm::MxType>(dtype), a);
    if (e != cudaSuccess) return fail_cuda(e, "mx_matmul launch");
    return Q4MM_OK;
}

int rope_rotate(const void *x, long long x_token_stride, long long x_head_stride, int dtype, const void *positions,
                int positions_64, const double *frequencies, int rotated, int interleaved, float magnitude, void *out,
                long long out_token_stride, long long out_head_stride, int tokens, int heads, int headDim,
                q4mm_stream_t stream) {
    int rc = check_mx_dtype(dtype, "input");
    if (rc) return rc;
    if (headDim <= 0 || headDim > Q4MM_ROPE_MAX_HEAD)
        return fail(Q4MM_ERR_DIM, "headDim (%d) must be between 1 and %d", headDim, Q4MM_ROPE_MAX_HEAD);
    if (heads <= 0 || heads > Q4MM_MX_MAX_HEADS)
        return fail(Q4MM_ERR_DIM, "heads (%d) must be between 1 and %d", heads, Q4MM_MX_MAX_HEADS);
    if (tokens < 0 || tokens > Q4MM_MX_MAX_ROWS)
        return fail(Q4MM_ERR_DIM, "tokens (%d) must be between 0 and %d", tokens, Q4MM_MX_MAX_ROWS);
    if (tokens == 0) return Q4MM_OK;
    if ((rc = check_rope(frequencies, rotated, magnitude, headDim)) ||
        (rc = check_head_strides(x_token_stride, x_head_stride, tokens, heads, headDim, false, "x")) ||
        (rc = check_head_strides(out_token_stride, out_head_stride, tokens, heads, headDim, true, "out")))
        return rc;
    const size_t size = mx_size(dtype), psize = positions_64 ? 8 : 4;
    const Span ins[3] = {head_span(x, x_token_stride, x_head_stride, tokens, heads, headDim, size, "x"),
                         Span{positions, (size_t)tokens * psize, "positions"},
                         Span{frequencies, (size_t)rotated / 2 * 8, "frequencies"}};
    const Span o = head_span(out, out_token_stride, out_head_stride, tokens, heads, headDim, size, "out");
    if ((rc = check_mx_ptr(ins[0], size)) || (rc = check_mx_ptr(ins[1], psize)) || (rc = check_mx_ptr(o, size)))
        return rc;
    const bool same = x == out && (tokens == 1 || x_token_stride == out_token_stride) &&
                      (heads == 1 || x_head_stride == out_head_stride);
    if ((rc = check_mx_alias(&o, 1, ins + (same ? 1 : 0), (same ? 1 : 2) + (rotated ? 1 : 0)))) return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx, false))) return rc;
    const q4mm::RopeArgs a{x, x_token_stride, x_head_stride, positions, positions_64 != 0,
                           q4mm::RopeView{frequencies, rotated, interleaved != 0, magnitude}, out, out_token_stride,
                           out_head_stride, tokens, heads, headDim};
    const cudaError_t e = q4mm::launch_rope_rotate(ctx, static_cast<q4mm::MxType>(dtype), a);
    if (e != cudaSuccess) return fail_cuda(e, "rope_rotate launch");
    return Q4MM_OK;
}

int mx_cache_write(const void *k, long long k_token_stride, long long k_head_stride, const void *v,
                   long long v_token_stride, long long v_head_stride, int dtype, const double *frequencies,
                   int rotated, int interleaved, float magnitude, void *k_codes, void *k_scales, void *v_codes,
                   void *v_scales, int pages, int kvHeads, int pageTokens, int headDim, int bits, const int *starts,
                   const int *lengths, const int *table, int sequences, int tableWidth, int tokens,
                   q4mm_stream_t stream) {
    CacheCall call{q4mm::MxCacheView{static_cast<uint8_t *>(k_codes), static_cast<uint8_t *>(k_scales),
                                     static_cast<uint8_t *>(v_codes), static_cast<uint8_t *>(v_scales), pages, kvHeads,
                                     pageTokens, headDim, bits},
                   q4mm::MxBatchView{starts, lengths, table, sequences, tableWidth}, {}};
    int rc = check_mx_dtype(dtype, "input");
    if (rc || (rc = check_cache(call, tokens)) || (rc = check_rope(frequencies, rotated, magnitude, headDim))) return rc;
    if (tokens == 0 || sequences == 0) return Q4MM_OK;
    if ((rc = check_head_strides(k_token_stride, k_head_stride, tokens, kvHeads, headDim, false, "k")) ||
        (rc = check_head_strides(v_token_stride, v_head_stride, tokens, kvHeads, headDim, false, "v")))
        return rc;
    const size_t size = mx_size(dtype);
    const Span ins[6] = {head_span(k, k_token_stride, k_head_stride, tokens, kvHeads, headDim, size, "k"),
                         head_span(v, v_token_stride, v_head_stride, tokens, kvHeads, headDim, size, "v"),
                         Span{frequencies, (size_t)rotated / 2 * 8, "frequencies"}, call.spans[4], call.spans[5],
                         call.spans[6]};
    if ((rc = check_mx_ptr(ins[0], size)) || (rc = check_mx_ptr(ins[1], size)) ||
        (rc = check_mx_alias(call.spans, 4, ins, 6)))
        return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx, false))) return rc;
    const q4mm::MxCacheIoArgs a{call.cache, call.batch, k, v, k_token_stride, k_head_stride, v_token_stride,
                                v_head_stride, tokens, ctx.status};
    const q4mm::RopeView rope{frequencies, rotated, interleaved != 0, magnitude};
    const cudaError_t e = q4mm::launch_mx_cache_write(ctx, static_cast<q4mm::MxType>(dtype), a, rope);
    if (e != cudaSuccess) return fail_cuda(e, "mx_cache_write launch");
    return Q4MM_OK;
}

int mx_cache_read(const void *k_codes, const void *k_scales, const void *v_codes, const void *v_scales, int pages,
                  int kvHeads, int pageTokens, int headDim, int bits, const int *starts, const int *lengths,
                  const int *table, int sequences, int tableWidth, void *k, long long k_token_stride,
                  long long k_head_stride, void *v, long long v_token_stride, long long v_head_stride, int dtype,
                  int tokens, q4mm_stream_t stream) {
    auto bytes = [](const void *p) { return const_cast<uint8_t *>(static_cast<const uint8_t *>(p)); };
    CacheCall call{q4mm::MxCacheView{bytes(k_codes), bytes(k_scales), bytes(v_codes), bytes(v_scales), pages, kvHeads,
                                     pageTokens, headDim, bits},
                   q4mm::MxBatchView{starts, lengths, table, sequences, tableWidth}, {}};
    int rc = check_mx_dtype(dtype, "output");
    if (rc || (rc = check_cache(call, tokens))) return rc;
    if (tokens == 0 || sequences == 0) return Q4MM_OK;
    if ((rc = check_head_strides(k_token_stride, k_head_stride, tokens, kvHeads, headDim, true, "k")) ||
        (rc = check_head_strides(v_token_stride, v_head_stride, tokens, kvHeads, headDim, true, "v")))
        return rc;
    const size_t size = mx_size(dtype);
    const Span outs[2] = {head_span(k, k_token_stride, k_head_stride, tokens, kvHeads, headDim, size, "k"),
                          head_span(v, v_token_stride, v_head_stride, tokens, kvHeads, headDim, size, "v")};
    if ((rc = check_mx_ptr(outs[0], size)) || (rc = check_mx_ptr(outs[1], size)) ||
        (rc = check_mx_alias(outs, 2, call.spans, 7)))
        return rc;
    q4mm::LaunchCtx ctx;
    if ((rc = device_ctx(stream, &ctx, false))) return rc;
    const q4mm::MxCacheIoArgs a{call.cache, call.batch, k, v, k_token_stride, k_head_stride, v_token_stride,
                                v_head_stride, tokens, ctx.status};
    const cudaError_t e = q4mm::launch_mx_cache_read(ctx, static_cast<q4mm::MxType>(dtype), a);
    if (e != cudaSuccess) return fail_cuda(e, "mx_cache_read launch");
    return Q4MM_OK;
}

int mx_attention(const void *q, long long q_token_stride, long long q_head_stride, int dtype, const void *k_codes,
                 const void *k_scales, const void *v_codes, const void *v_scales, int pages, int kvHeads,
                 int pageTokens, int headDim, int bits, const int *starts, const int *lengths, const int *table,
                 int sequences, int tableWidth, float scale, int causal, void *y, long long y_token_stride,
                 long long y_head_stride, int tokens, int heads, void *workspace, size_t workspace_bytes,
                 q4mm_stream_t stream) {
    auto bytes = [](const void *p) { return const_cast<uint8_t *>(static_cast<const uint8_t *>(p)); };
    CacheCall call{q4mm::MxCacheView{bytes(k_codes), bytes(k_scales), bytes(v_codes), bytes(v_scales), pages, kvHeads,
                                     pageTokens, headDim, bits},
                   q4mm::MxBatchView{starts, lengths, table, sequences, tableWidth}, {}};
    int rc = check_mx_dtype(dtype, "input");
    if (rc || (rc = check_cache(call, tokens))) return rc;
    if (heads <= 0 || heads > Q4MM_MX_MAX_HEADS || heads % kvHeads)
        return fail(Q4MM_ERR_DIM, "heads (%d) must be a positive multiple of kvHeads (%d), at most %d", heads, kvHeads,
                    Q4MM_MX_MAX_HEADS);
    if ((rc = check_rows(tokens, heads / kvHeads))) return rc;
    if (!(scale >= 0.f && scale - scale == 0.f)) return fail(Q4MM_ERR_DIM, "scale (%g) must be finite and not negative", (double)scale);
    if (tokens == 0 || sequences == 0) return Q4MM_OK;
    if ((rc = check_head_strides(q_token_stride, q_head_stride, tokens, heads, headDim, false, "q")) ||
        (rc = check_head_strides(y_token_stride, y_head_stride, tokens, heads, headDim, true, "y")))
        return rc;
    const size_t size = mx_size(dtype);
    const Span qs = head_span(q, q_token_stride, q_head_stride, tokens, heads, headDim, size, "q");
    const Span ys = head_span(y, y_token_stride, y_head_stride, tokens, heads, headDim, size, "y");
    if ((rc = check_mx_ptr(qs, size)) || (rc = check_mx_ptr(ys, size)) || (rc = check_mx_alias(&ys, 1, &qs, 1)) ||
        (rc = check_mx_alias(&ys, 1, call.spans, 7)))
        return rc;
    if (workspace_bytes) {
        const Span ws{workspace, workspace_bytes, "workspace"};
        if ((rc = check_mx_ptr(ws, 16)) || (rc = check_mx_alias(&ws, 1, call.spans, 7)) ||
            (rc = check_mx_alias(&ws, 1, &qs, 1)) || (rc = check_mx_alias(&ws, 1, &ys, 1)))
            return rc;
    }
    q4mm::LaunchCtx ctx;
    const bool vec = reinterpret_cast<uintptr_t>(q) % (4 * size) == 0 && reinterpret_cast<uintptr_t>(y) % (4 * size) == 0 &&
                     q_token_stride % 4 == 0 && q_head_stride % 4 == 0 && y_token_stride % 4 == 0 &&
                     y_head_stride % 4 == 0;
    if ((rc = device_ctx(stream, &ctx, false))) return rc;
    q4mm::AttentionPlan plan = plan_attention(tokens, heads, kvHeads, sequences, tableWidth, pageTokens, dtype, ctx.num_sms);
    if (!plan.many && plan.few.parts > 1) {  // as many parts as the workspace holds
        const size_t all = q4mm::mx_attention_few_workspace(tokens, heads, kvHeads, headDim, sequences, plan.few);
        const size_t held = workspace_bytes / (all / plan.few.parts);
        if (held < (size_t)plan.few.parts) plan.few.parts = held ? (int)held : 1;
        plan.few_as_f32 |= q4mm::few_chain_passes(q4mm::table_keys(tableWidth, pageTokens), plan.few, attention_chain(dtype));
    }
    if (plan.many) take_fault(&ctx);
    const q4mm::MxAttentionArgs a{call.cache, call.batch, q, q_token_stride, q_head_stride, y, y_token_stride,
                                  y_head_stride, scale, causal != 0, tokens, heads, static_cast<q4mm::MxType>(dtype),
                                  vec, static_cast<float *>(workspace), workspace_bytes, ctx.status};
    const cudaError_t e =
        plan.many ? q4mm::launch_mx_attention_many(ctx, a, plan.split, plan.many_as_f32)
                  : q4mm::launch_mx_attention_few(ctx, a, plan.few, plan.few_as_f32);
    if (e != cudaSuccess) return fail_cuda(e, "mx_attention launch");
    return Q4MM_OK;
}

size_t mx_attention_workspace(int kvHeads, int pageTokens, int headDim, int sequences, int tableWidth, int tokens,
                              int heads) {
    if (kvHeads <= 0 || heads <= 0 || heads % kvHeads || pageTokens <= 0 || sequences <= 0 || tableWidth < 0 || tokens <= 0 ||
        (long long)tokens * (heads / kvHeads) > Q4MM_MX_MAX_ROWS)
        return 0;
    q4mm::LaunchCtx ctx;
    if (device_ctx(nullptr, &ctx, false)) return 0;
    size_t most = 0;
    for (const int dtype : {Q4MM_F32, Q4MM_F16, Q4MM_BF16}) {
        const q4mm::AttentionPlan plan =
            plan_attention(tokens, heads, kvHeads, sequences, tableWidth, pageTokens, dtype, ctx.num_sms);
        const size_t bytes =
            plan.many ? 0 : q4mm::mx_attention_few_workspace(tokens, heads, kvHeads, headDim, sequences, plan.few);
        if (bytes > most) most = bytes;
    }
    return most;
}

int q4mm_call(int which, const long long *w) {
    auto p = [&](int i) { return reinterpret_cast<void *>(w[i]); };
    auto ints = [&](int i) { return reinterpret_cast<const int *>(w[i]); };
    auto real = [&](int i) {
        double d;
        memcpy(&d, w + i, sizeof(d));
        return (float)d;
    };
    auto i32 = [&](int i) { return (int)(w[i] > 0x7FFFFFFF ? 0x7FFFFFFF : w[i] < -1 ? -1 : w[i]); };
    auto stream = [&](int i) { return reinterpret_cast<q4mm_stream_t>(w[i]); };
    if (!w) return fail(Q4MM_ERR_NULL, "the words of a call must be non-NULL");
    switch (which) {
        case Q4MM_CALL_ROPE_ROTATE:
            return rope_rotate(p(0), w[1], w[2], i32(3), p(4), i32(5), static_cast<const double *>(p(6)), i32(7), i32(8),
                               real(9), p(10), w[11], w[12], i32(13), i32(14), i32(15), stream(16));
        case Q4MM_CALL_MX_CACHE_WRITE:
            return mx_cache_write(p(0), w[1], w[2], p(3), w[4], w[5], i32(6), static_cast<const double *>(p(7)), i32(8),
                                  i32(9), real(10), p(11), p(12), p(13), p(14), i32(15), i32(16), i32(17), i32(18), i32(19),
                                  ints(20), ints(21), ints(22), i32(23), i32(24), i32(25), stream(26));
        case Q4MM_CALL_MX_CACHE_READ:
            return mx_cache_read(p(0), p(1), p(2), p(3), i32(4), i32(5), i32(6), i32(7), i32(8), ints(9), ints(10), ints(11),
                                 i32(12), i32(13), p(14), w[15], w[16], p(17), w[18], w[19], i32(20), i32(21), stream(22));
        case Q4MM_CALL_MX_ATTENTION:
            return mx_attention(p(0), w[1], w[2], i32(3), p(4), p(5), p(6), p(7), i32(8), i32(9), i32(10), i32(11), i32(12),
                                ints(13), ints(14), ints(15), i32(16), i32(17), real(18), i32(19), p(20), w[21], w[22],
                                i32(23), i32(24), p(25), (size_t)w[26], stream(27));
    }
    return fail(Q4MM_ERR_DIM, "there is no call %d", which);
}

const char *q4mm_last_error(void) { return g_err; }

int q4mm_device_status(q4mm_stream_t stream, int clear) {
    q4mm::LaunchCtx ctx;
    int rc = device_ctx(stream, &ctx, false);
    if (rc) return rc;
    int host = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(&host, ctx.status, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return fail_cuda(e, "reading the device status word");
    if (clear && host) {
        const int zero = 0;
        e = cudaMemcpyAsync(ctx.status, &zero, sizeof(int), cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) return fail_cuda(e, "clearing the device status word");
    }
    if (host & q4mm::kStatusTimeout)
        return fail(Q4MM_ERR_TIMEOUT, "a bounded in-kernel wait ran out (status word %d)", host);
    if (host) return fail(Q4MM_ERR_INDEX, "a call met a page number or a position outside its cache or table");
    return Q4MM_OK;
}

int q4mm_test_fail_next_wait(int stage, long long limit_cycles) {
    if (stage == -1) {
        g_test_fault.armed = false;
        return Q4MM_OK;
    }
    if (stage < 0 || limit_cycles <= 0)
        return fail(Q4MM_ERR_DIM, "q4mm_test_fail_next_wait: stage (%d) must be >= 0 (or -1) and limit (%lld) > 0",
                    stage, limit_cycles);
    g_test_fault.armed = true;
    g_test_fault.stage = stage;
    g_test_fault.limit = limit_cycles;
    return Q4MM_OK;
}

int q4mm_test_attention_kernel(int which) {
    if (which < 0 || which > 2) return fail(Q4MM_ERR_DIM, "q4mm_test_attention_kernel: %d must be 0, 1 or 2", which);
    g_test_attention = which;
    return Q4MM_OK;
}

int q4mm_version(void) { return 400; }

}  // extern "C"

/*
 * q4mm — GB300 (sm_103a) kernels for the Linear-layer product y = x·Wᵀ with
 * an FP32 activation and a block-quantized weight that is dequantized inside
 * the kernel.  C ABI of libq4mm.so.
 *
 * Shapes and layouts (every entry point):
 *   K = inputDim, N = outputDim, T = tokens.
 *   x  : T rows of K fp32 values, row-major ([T][K]); token r starts at x + r·K.
 *   W  : N output rows stored one after another ([out, in] order, used in
 *        place, never transposed; SKaiNET docs "Eager execution: backends and
 *        kernels", paragraph on the dense x·Wᵀ row).  Each row is a run of
 *        contiguous blocks (the BLOCKED_ROW_MAJOR order of SKaiNET issue
 *        #1138, section "Tasks").
 *   y  : T rows of N fp32 values, row-major ([T][N]); token r writes y + r·N
 *        (the prefill loop "advance offsets by r·k / r·n", same section).
 *        y is overwritten, never accumulated into.
 *
 * Ownership and memory: x, W and y are DEVICE pointers owned by the caller
 * and must not overlap.  q4k_matmul and ternary_gemv allocate nothing;
 * q4k_matmul_tc takes stream-ordered scratch for the length of each call
 * above 128 tokens (its entry below gives the size).
 *
 * Streams: every compute call is asynchronous on `stream` (NULL means the
 * legacy default stream).  Validation is synchronous: an invalid call returns
 * its error before anything is launched and leaves y untouched.  Calls on one
 * stream may overlap their prologue with the previous kernel on that stream
 * (programmatic dependent launch): weight bytes, which no earlier kernel
 * writes, may be fetched before the previous kernel has finished; x is read
 * and y written only after it has.
 *
 * Device: a call runs on the current device (cudaGetDevice), whose pointers
 * and stream it must be given.
 *
 * Errors: every entry point returns Q4MM_OK (0) or a negative q4mm_status;
 * q4mm_last_error() then returns a message for the calling thread.  No C++
 * exception crosses this boundary.  Asynchronous faults surface through the
 * CUDA runtime as usual (the next synchronising call on the stream).
 */
#ifndef Q4MM_H
#define Q4MM_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as the CUDA runtime's cudaStream_t. */
struct CUstream_st;
typedef struct CUstream_st *q4mm_stream_t;

typedef enum {
    Q4MM_OK = 0,
    Q4MM_ERR_DIM = -1,     /* a dimension is <= 0, above its limit, or inputDim breaks its multiple */
    Q4MM_ERR_NULL = -2,    /* a required pointer is NULL */
    Q4MM_ERR_ALIGN = -3,   /* a pointer is not aligned as its entry point requires */
    Q4MM_ERR_CUDA = -4,    /* the CUDA runtime reported an error (launch, device query) */
    Q4MM_ERR_TIMEOUT = -5, /* a bounded in-kernel wait ran out (see q4mm_device_status) */
    Q4MM_ERR_ALIAS = -6,   /* x, W and y overlap */
    Q4MM_ERR_INDEX = -7    /* a page number or position outside the cache (see q4mm_device_status) */
} q4mm_status;

/* Largest inputDim accepted by every entry point. */
#define Q4MM_MAX_INPUT_DIM 65536

/*
 * q4k_matmul — y = x·Wᵀ with W in Q4_K, FP32 arithmetic.
 *
 * Defined by SKaiNET PR #562 "feat(kernel): SIMD-fused Q4_K matmul kernel +
 * Q4KMatmulKernel SPI": section "Pipeline" (the 256-value super-block, the
 * strided nibble layout with sub-block 2j in the low nibbles and 2j+1 in the
 * high nibbles of the same 32 bytes, value = d·sc·q − dmin·m, and the lazy
 * correction acc += scale·codeSum − offset·inputSum) and section "Test plan"
 * (inputDim must be a multiple of 256; results within 1e-4 relative of the
 * dequantize-then-matmul reference).
 *
 * w_q4k : N·(K/256) blocks of 144 bytes: fp16 d (little-endian), fp16 dmin,
 *         12 bytes packing eight 6-bit scales and eight 6-bit mins (ggml
 *         canonical packing), 128 bytes of 4-bit codes.  16-byte aligned.
 * x     : 16-byte aligned.  y: 4-byte aligned.
 * Limits: inputDim a positive multiple of 256 and <= Q4MM_MAX_INPUT_DIM;
 *         outputDim >= 1; tokens >= 1.
 * Precision: per token row t, max_o |y − y_exact| <= 1e-4 · max_o |y_exact|
 *         on the pages' test inputs and on rows with a wide dynamic range
 *         (activations of 1e5 next to ones of order 1, including on weights
 *         that are zero).  The bound behind it, up to 2 tokens: each 32-value
 *         group g of x is rounded once to a multiple of s_g·2^-23, s_g the
 *         power of two just above max_g|x|/255, i.e. to within
 *         max(2^-23·max_g|x|/255, 2^-127) (about 4.7e-10 of the group's
 *         largest magnitude; values within a factor 255 of it are exact),
 *         split into four byte planes, and the code-dots are exact integer
 *         sums; so |y_o − y_exact,o| <= Σ_g 2^-23·max_g|x|/255·Σ_{k∈g}|w_ok|
 *         plus fp32 rounding of the scales, mins and sums (relative 2^-22 or
 *         so of each term).  A large activation changes only its own group's
 *         grid.  Where that kernel's geometry does not fit (2 tokens with a
 *         large inputDim), and from 3 tokens on: fp32 dequantization and fp32
 *         fused multiply-add.
 * Weights are streamed from HBM once per call for up to 8 tokens; above
 * that once per 8 tokens (up to 32 tokens, or whenever outputDim is below
 * about 6,500 rows) or once per 64 tokens (the FP32 tile kernel).
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int q4k_matmul(const float *x, const void *w_q4k, float *y, int inputDim, int outputDim,
               int tokens, q4mm_stream_t stream);

/*
 * q4k_matmul_tc — the same product on the tensor cores (tcgen05), for
 * prefill-sized token counts.  The dequantized weight (computed in fp32 and
 * rounded once) and the activation are rounded to bfloat16 before the
 * multiply; products are accumulated in FP32 (tensor memory).  Same layouts,
 * alignment and limits as q4k_matmul.
 * Precision: per token row, max_o |y − y_bf16| <= 1e-4 · max_o |y_bf16| where
 * y_bf16 is the exact product of the bf16-rounded operands; the deviation
 * from the exact product is that of bf16 operand rounding (about 5e-3 of
 * max_o |y_exact| on random data).
 * Memory: up to 128 tokens a call allocates nothing (the kernel rounds x to
 * bf16 as it loads it).  Above 128 tokens each call takes stream-ordered
 * scratch (cudaMallocAsync on `stream`, released by cudaFreeAsync on
 * `stream` after the call's last kernel): the bf16 copy of x,
 * 2·tokens·inputDim bytes rounded up to 256, and the weights are read once
 * per 128 tokens.  The S = max(3, ceil(inputDim/16384)) CTAs of a cluster
 * that split the input dimension of each 256-row tile add their partial
 * sums in shared memory.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA} (CUDA also when the
 * scratch allocation fails).  A bounded wait that runs out sets the device
 * status word (see q4mm_device_status).
 */
int q4k_matmul_tc(const float *x, const void *w_q4k, float *y, int inputDim, int outputDim,
                  int tokens, q4mm_stream_t stream);

/* Largest inputDim accepted by q4_0_gemv. */
#define Q4MM_Q4_0_MAX_INPUT_DIM 32768

/*
 * q4_0_gemv — y = x·Wᵀ with W in Q4_0, FP32 result.
 *
 * The block is the one SKaiNET PR #562 names as its follow-up (section "Out
 * of scope": Q4_0, "same algorithm, simpler block", 32 values in 18 bytes).
 * The page gives no byte layout; this library reads it as ggml's: fp16 d
 * (little-endian), then 16 bytes qs; element l (l < 16) of a block is the low
 * nibble of qs[l] and element 16 + l its high nibble (the same strided
 * pattern as the Q4_K slabs); w = d·(q − 8), i.e. scale d and offset 8·d in
 * the page's lazy form.
 *
 * w_q4_0 : N·(K/32) blocks of 18 bytes, each row contiguous.  16-byte aligned.
 * x      : 16-byte aligned.  y: 4-byte aligned.
 * Limits: inputDim a positive multiple of 256 and <= Q4MM_Q4_0_MAX_INPUT_DIM
 *         (the one-token kernel's geometry: 256 values occupy 144 bytes of a
 *         row, as in Q4_K); outputDim >= 1; tokens >= 1.
 * Precision: as the one-token path of q4k_matmul: per token row,
 *         max_o |y − y_exact| <= 1e-4 · max_o |y_exact|, with x rounded once
 *         to within 2^-23/255 of each 32-value group's largest magnitude and
 *         the code-dots exact integer sums of (q − 8)·x̂, so a zero weight
 *         (q = 8) adds nothing whatever its activation.
 * Tokens: up to 8 tokens share one pass over the weights (more tokens
 *         take one pass per 8).
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int q4_0_gemv(const float *x, const void *w_q4_0, float *y, int inputDim, int outputDim,
              int tokens, q4mm_stream_t stream);

/* Largest inputDim accepted by q6k_gemv. */
#define Q4MM_Q6K_MAX_INPUT_DIM 32768

/*
 * q6k_gemv — y = x·Wᵀ with W in Q6_K, FP32 result.
 *
 * The block is the second follow-up SKaiNET PR #562 names (section "Out of
 * scope": Q6_K, "ql + qh with the 4-codes-per-qh-byte half-interleaved
 * layout").  The page gives no byte layout; this library reads it as ggml's:
 * 256 values in 210 bytes — ql[128] (low 4 bits of each 6-bit code), qh[64]
 * (high 2 bits, four codes per byte), 16 signed 8-bit sub-block scales, fp16
 * d (little-endian) last.  In half n (values 128n..128n+127), value
 * 128n + 32g + l (g = 0..3, l < 32) takes the low nibble of ql[64n + l]
 * (g = 0) or of ql[64n + 32 + l] (g = 1), the high nibble of ql[64n + l]
 * (g = 2) or of ql[64n + 32 + l] (g = 3), and bits 2g..2g+1 of qh[32n + l];
 * its sub-block is 8n + 2g + l/16 and w = d·scale·(q − 32).
 *
 * w_q6k : N·(K/256) blocks of 210 bytes, each row contiguous (rows need not
 *         start on a 16-byte boundary).  The buffer is 16-byte aligned.
 * x     : 16-byte aligned.  y: 4-byte aligned.
 * Limits: inputDim a positive multiple of 256 and <= Q4MM_Q6K_MAX_INPUT_DIM;
 *         outputDim >= 1; tokens >= 1 (up to 8 tokens per pass over the
 *         weights).
 * Precision: as the one-token path of q4k_matmul: per token row,
 *         max_o |y − y_exact| <= 1e-4 · max_o |y_exact|; the code-dots are
 *         exact integer sums of (q − 32)·x̂, so a zero weight adds nothing.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int q6k_gemv(const float *x, const void *w_q6k, float *y, int inputDim, int outputDim, int tokens,
             q4mm_stream_t stream);

/* Largest inputDim accepted by q4k_ffn_swiglu. */
#define Q4MM_FFN_MAX_INPUT_DIM 32768

/*
 * q4k_ffn_swiglu — the input side of a Llama feed-forward block in one call:
 *   h = silu(x·W_gateᵀ) ⊙ (x·W_upᵀ),  silu(z) = z / (1 + e^(−z)),
 * both weights Q4_K (layout, values and precision as q4k_matmul's: the
 * byte-plane path for 1-2 tokens, fp32 FMA from 3 tokens on).  The pages
 * name this fused operation only as the llama.cpp benchmark "ffn_swiglu"
 * (PR #37 "ggml-cpu: cache-aware tiling in ggml_compute_forward_mul_mat",
 * section "Measured impact"); the formula is the standard Llama FFN.  For
 * 1-2 tokens one launch per token, from 3 tokens on one launch per 8 tokens,
 * each reading x once for both weights and writing only h.
 *
 * w_gate, w_up : hiddenDim rows of inputDim/256 Q4_K blocks each, 16-byte
 *                aligned; they may be the same buffer.  x: 16-byte aligned.
 *                h: [tokens][hiddenDim], 4-byte aligned, overwritten; h must
 *                not overlap x or either weight.
 * Limits: inputDim a positive multiple of 256 and <= Q4MM_FFN_MAX_INPUT_DIM;
 *         hiddenDim >= 1; tokens >= 1 (one pass over both weights per token
 *         up to 2 tokens, per 8 tokens above).
 * Precision: g and u each within q4k_matmul's bound; h = silu(g)·u
 *         in fp32 (expf), so max_o |h − h_exact| <= 1e-4 · max_o |u| ·
 *         (1.1 · max_o |g| + max_o |silu(g)|) per token (1.1 bounds |silu'|).
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int q4k_ffn_swiglu(const float *x, const void *w_gate, const void *w_up, float *h, int inputDim,
                   int hiddenDim, int tokens, q4mm_stream_t stream);

/* Size of the fixed device array that q4k_matmul_tc_noalloc uses as scratch. */
#define Q4MM_TC_NOALLOC_SCRATCH_BYTES (16u << 20)

/*
 * q4k_matmul_tc_noalloc — q4k_matmul_tc with no allocation at all.  The pages
 * that define the product have no counterpart of this entry point.  It is for
 * callers that cannot allocate device memory while a call runs: a host
 * framework whose own allocator owns the whole device budget and forbids
 * allocations behind its back, a process on a device or driver set-up
 * without stream-ordered memory pools (where cudaMallocAsync fails), or a
 * serving loop with a latency budget that keeps allocator calls off its hot
 * path.
 *
 * Same arguments, layouts, alignment, limits, precision and results as
 * q4k_matmul_tc: the same kernels run.  The scratch that q4k_matmul_tc takes
 * per call lives instead in one fixed array of Q4MM_TC_NOALLOC_SCRATCH_BYTES
 * (16 MiB) of device memory inside the library, which every GPU that loads
 * the library holds until the process exits.  A call whose scratch (the size
 * formula under q4k_matmul_tc) is larger returns Q4MM_ERR_DIM before
 * launching anything; calls of up to 128 tokens need none, 256 tokens of a
 * 4096 → 11008 layer need 2 MiB, and the array holds up to 2048 tokens at
 * inputDim 4096.
 *
 * Sharing: every call on a device uses the same array, which keeps the last
 * call's contents.  No part of it has to start at zero: a call writes every
 * byte of scratch before reading it.  Calls whose kernels may overlap on the
 * GPU (different streams with no ordering between them, or several host
 * threads) race on the array: issue them on one stream or synchronise
 * between them.
 *
 * Set-up: the first call on each device, with that device current, looks up
 * the array's device address (cudaGetSymbolAddress) and keeps it for later
 * calls; make that first call before any stream capture.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int q4k_matmul_tc_noalloc(const float *x, const void *w_q4k, float *y, int inputDim,
                          int outputDim, int tokens, q4mm_stream_t stream);

/* Bytes per row and 64-value chunk of the relayouted tensor-core layout, rows
 * per tile, and the size of a relayouted inputDim → outputDim weight (rows
 * rounded up to whole tiles). */
#define Q4MM_TC_CHUNK_BYTES 48
#define Q4MM_TC_TILE_ROWS 256
#define Q4MM_TC_RELAYOUT_BYTES(inputDim, outputDim)                                                \
    (((size_t)(outputDim) + Q4MM_TC_TILE_ROWS - 1) / Q4MM_TC_TILE_ROWS * Q4MM_TC_TILE_ROWS *        \
     (size_t)((inputDim) / 64) * Q4MM_TC_CHUNK_BYTES)

/*
 * q4k_relayout_tc — the one-time relayout of a Q4_K weight for
 * q4k_matmul_tc_relayouted: done once when the weight is registered, not on
 * every call (SKaiNET docs "Eager execution: backends and kernels", the
 * paragraph on weights relayouted once rather than per call; the page names
 * no target layout, so this one is the library's own).
 *
 * Layout written to w_tc.  Each 64-value chunk c of a row (values
 * 64c..64c+63: the slab j = c mod 4 of block b = c/4, its 32 code bytes
 * qs[32j..32j+31], low nibbles = sub-block 2j, high nibbles = 2j+1) becomes
 * 48 bytes:
 *   bytes  0..3  fp32 d·sc(2j)      bytes  4..7  fp32 dmin·m(2j)
 *   bytes  8..11 fp32 d·sc(2j+1)    bytes 12..15 fp32 dmin·m(2j+1)
 *   bytes 16..47 the 32 code bytes, unchanged
 * (floats little-endian).  Rows are grouped in tiles of Q4MM_TC_TILE_ROWS
 * (256), the last tile padded with zero rows, and stored tile-major: chunk c
 * of the 256 rows of tile t is one contiguous run of 256·48 bytes at byte
 * (t·(inputDim/64) + c)·12288, row r of the tile at 48·r within it.  The
 * tensor-core kernel then fetches each chunk of a tile with one plain bulk
 * copy.  Every product is exact in fp32, so the relayouted weight
 * dequantizes to the same fp32 matrix (w = scale·q − offset), and
 * q4k_matmul_tc_relayouted gives bit for bit the result of q4k_matmul_tc on
 * the canonical weight.  The layout keeps products, not factors: it cannot
 * be turned back into the canonical bytes.  It is about 4/3 the size of the
 * canonical weight (0.75·inputDim bytes per row, plus padding rows, against
 * 0.5625·inputDim).
 *
 * Arguments: w_q4k (device, read) the canonical weight, outputDim rows of
 * inputDim/256 blocks of 144 bytes; w_tc (device, written, padding rows
 * included) a buffer of Q4MM_TC_RELAYOUT_BYTES(inputDim, outputDim) bytes
 * owned by the caller.  Both 16-byte aligned, not overlapping; inputDim a
 * positive multiple of 256 up to Q4MM_MAX_INPUT_DIM, outputDim positive.
 * Asynchronous on `stream`; allocates nothing.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int q4k_relayout_tc(const void *w_q4k, void *w_tc, int inputDim, int outputDim, q4mm_stream_t stream);

/*
 * q4k_matmul_tc_relayouted — q4k_matmul_tc on a weight made by
 * q4k_relayout_tc: the same kernels, tiles, precision, scratch and results
 * (bit for bit); the dequantizing warps read the two sub-block scales of a
 * chunk as ready fp32 values instead of decoding the 6-bit scale field.
 * w_tc: Q4MM_TC_RELAYOUT_BYTES(inputDim, outputDim) bytes as q4k_relayout_tc
 * wrote them, 16-byte aligned.  Everything else as q4k_matmul_tc.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int q4k_matmul_tc_relayouted(const float *x, const void *w_tc, float *y, int inputDim, int outputDim,
                             int tokens, q4mm_stream_t stream);

/*
 * ternary_gemv — y = scale · (x·codesᵀ) with W in the BitNet b1.58 payload.
 *
 * Defined by SKaiNET issue #1138 "[ternary-f32] Phase 2: TernaryF32GemvNative
 * SPI + reference ViewKernel + TernaryF32KernelPack", section "Tasks": four
 * codes per byte, code(o, i) = ((byte >> 2·(i%4)) & 3) − 1 for byte
 * o·K/4 + i/4; out[o] = Σ_k in[k]·code(o,k) accumulated in FP32; the scale
 * multiplies the finished dot product once (pass 1.0f for the seam's raw,
 * unscaled code-dot); rows for prefill advance by r·k and r·n.
 *
 * w_packed : N rows of K/4 bytes, no alignment required.  x: 16-byte
 *            aligned.  y: 4-byte aligned.
 * Limits: inputDim a positive multiple of 4 and <= Q4MM_MAX_INPUT_DIM;
 *         outputDim >= 1; tokens >= 1.
 * Precision: FP32.  The field value 3 decodes to +2 by the literal formula.
 *            With integer activations the code-dot is exact, so y equals
 *            the single fp32 rounding of scale × dot bit for bit.  Up to 3
 *            tokens with inputDim a multiple of 256 (and W 16-byte aligned)
 *            x is split as in q4k_matmul's one-token path and the code-dot
 *            is an exact integer sum of code·x̂.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int ternary_gemv(const float *x, const void *w_packed, float scale, float *y, int inputDim,
                 int outputDim, int tokens, q4mm_stream_t stream);

/*
 * ---- Microscaled (MX) tensors --------------------------------------------
 *
 * The block formats of the OCP Microscaling Formats (MX) specification 1.0:
 * `rows` vectors of K values in blocks of 32 along K.  A block has one scale
 * 2^(b - 127), kept as the byte b (E8M0; 255 stands for NaN), and 32 codes in
 * `bits` bits:
 *   4: E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two codes to a
 *      byte, the even value in the low nibble;
 *   8: E4M3 (largest magnitude 448).
 * A value is its code times its block's scale.
 *
 * Layout.  K is padded with zero codes to Kp, the next multiple of 128.
 *   codes : rows of Kp·bits/8 bytes one after another (32-byte aligned base).
 *   scales: tiles of 128 rows x 4 blocks, 512 bytes each; tile (i, j) holds
 *           rows 128·i .. and blocks 4·j .. and lies at 512·(i·Kp/128 + j);
 *           in it the byte of (row r, block b) is
 *           16·(r % 32) + 4·(r % 128 / 32) + b % 4 (16-byte aligned base).
 *           Bytes of padding rows and blocks are written as zero by the
 *           quantising calls; a user's own layout must not put 255 there for
 *           padding blocks (codes zero times NaN is NaN).
 *
 * Quantisation of a block v: with amax = max |v|, the scale is
 * 2^(floor(log2 amax) - emax), emax = 2 (4 bits) or 8 (8 bits), at least
 * 2^-127 (amax = 0 gives byte 0); a code is v / scale (exact) rounded to
 * nearest even and cut at the largest code.  A block that holds an infinity
 * or a NaN gets scale NaN and zero codes: all 32 values become NaN.
 *
 * Element types of the other side are named by a q4mm_dtype.  Rows of those
 * tensors may be strided (in elements, the values of a row adjacent); any
 * base aligned to its element is accepted.  Accesses are fastest where every
 * row starts on a multiple of eight values in memory and K is a multiple of 8;
 * elsewhere up to 15 bytes between two rows of an input may be read with them
 * (never before the first row or past the last), and are not used.
 *
 * rows = 0 (tokens = 0) is a call with nothing to do and returns Q4MM_OK.
 * Every operand, weights included, may have been written by the previous
 * kernel on the stream.  No call allocates, and nothing persists.
 */
typedef enum { Q4MM_F32 = 0, Q4MM_F16 = 1, Q4MM_BF16 = 2 } q4mm_dtype;

/* Largest rows, tokens and outputDim of an MX call (indexes stay in an int). */
#define Q4MM_MX_MAX_ROWS 0x7FFFFE00

#define Q4MM_MX_PADDED(K) (((size_t)(K) + 127) / 128 * 128)
#define Q4MM_MX_CODE_BYTES(K, rows, bits) ((size_t)(rows) * (Q4MM_MX_PADDED(K) * (bits) / 8))
#define Q4MM_MX_SCALE_BYTES(K, rows) (((size_t)(rows) + 127) / 128 * (Q4MM_MX_PADDED(K) / 128) * 512)

/*
 * mx_quantize — x [rows][K] of type dtype to MX codes and scales.
 * codes: Q4MM_MX_CODE_BYTES(K, rows, bits); scales: Q4MM_MX_SCALE_BYTES(K, rows).
 * Limits: 1 <= inputDim <= Q4MM_MAX_INPUT_DIM; 0 <= rows <= Q4MM_MX_MAX_ROWS;
 *         bits 4 or 8.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int mx_quantize(const void *x, long long x_stride, int dtype, void *codes, void *scales, int inputDim, int rows,
                int bits, q4mm_stream_t stream);

/*
 * mx_swiglu — silu(gate)·up quantised as by mx_quantize, in one pass:
 * gate / (1 + e^-gate) · up in fp32, rounded once, to codes.  gate and up
 * may be two parts of one tensor's rows.  The value before its rounding is
 * within 10·2^-24 of the exact one (and 2^-149), also where e^-gate itself is
 * beyond fp32; gate = -infinity gives NaN, as the formula does.
 * Limits and returns as mx_quantize.
 */
int mx_swiglu(const void *gate, long long gate_stride, const void *up, long long up_stride, int dtype, void *codes,
              void *scales, int hiddenDim, int rows, int bits, q4mm_stream_t stream);

/*
 * mx_rmsnorm — the residual's addition, the RMS norm and its quantisation:
 *   h = x + residual                       (residual NULL: h = x)
 *   v = h · (mean_k h² + eps)^-1/2 · weight
 * in fp32; v is quantised as by mx_quantize, and h is written in x's type
 * where h is not NULL (the norm takes it before that rounding).  h may be x
 * or residual itself (same base and stride), and overlaps nothing else.
 * weight: K values of x's type or of Q4MM_F32.  The sum of squares is an
 * fp32 sum in a fixed order; it overflows where h reaches about 1e19, and with
 * eps = 0 a row whose squares all underflow (|h| below about 1e-23) is NaN.
 * Limits and returns as mx_quantize, and eps >= 0.
 */
int mx_rmsnorm(const void *x, long long x_stride, const void *residual, long long residual_stride, void *h,
               long long h_stride, int dtype, const void *weight, int weight_dtype, float eps, void *codes,
               void *scales, int inputDim, int rows, int bits, q4mm_stream_t stream);

/*
 * mx_dequantize — the values an MX tensor stands for, y [rows][K] of type
 * dtype (exact in fp32; else rounded once).  Limits and returns as mx_quantize.
 */
int mx_dequantize(const void *codes, const void *scales, void *y, long long y_stride, int dtype, int inputDim,
                  int rows, int bits, q4mm_stream_t stream);

/*
 * mx_matmul — y = x·Wᵀ on the tensor cores, x an MX tensor of `tokens` rows in
 * x_bits (4 or 8) bits, W one of outputDim rows in 4 bits, both over inputDim
 * values.  Products of codes and scales are exact; they are added in fp32.
 * y: [tokens][outputDim] of type dtype, contiguous, overwritten, aligned to
 * its element.
 * Limits: 1 <= inputDim <= Q4MM_MAX_INPUT_DIM; 1 <= outputDim <=
 *         Q4MM_MX_MAX_ROWS; 0 <= tokens <= Q4MM_MX_MAX_ROWS.
 * Precision: |y − y_exact| <= (K/32 + 1)·2^-23·Σ|x·w| before the rounding to
 *         dtype; the same call gives the same bits again.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int mx_matmul(const void *x_codes, const void *x_scales, int x_bits, const void *w_codes, const void *w_scales,
              void *y, int dtype, int inputDim, int outputDim, int tokens, q4mm_stream_t stream);

/*
 * ---- Attention on a paged MX cache ----------------------------------------
 *
 * rope_rotate — rotary positions.  x [tokens][heads][headDim] of type dtype,
 * strides in elements, the values of a head adjacent.  The first `rotated`
 * values of a head (an even number) are pairs (u, v), (2i, 2i + 1) where
 * interleaved, else (i, i + rotated / 2); with a = position · frequencies[i]
 *   u' = magnitude · (u cos a − v sin a),  v' = magnitude · (v cos a + u sin a)
 * and the values behind them are copied.  out is x itself (same base and
 * strides) or does not overlap it.
 * positions: `tokens` values of 32 bits, or of 64 where positions_64; any
 *            sign.  frequencies: rotated / 2 doubles, radians per position
 *            (NULL where rotated is 0).  The angle is reduced exactly; the
 *            frequency is taken to 2^-61 radians (and 2^-60 of itself), so
 *            an angle is off by that times the position.
 * Precision: fp32; cos and sin within 2·2^-24, so |u' − exact| <=
 *            2^-22·magnitude·(|u| + |v|) before the rounding to dtype.
 * Limits: 1 <= headDim <= Q4MM_ROPE_MAX_HEAD; 0 <= rotated <= headDim, even;
 *         1 <= heads <= Q4MM_MX_MAX_HEADS; 0 <= tokens <=
 *         Q4MM_MX_MAX_ROWS; magnitude finite.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
#define Q4MM_ROPE_MAX_HEAD 256
#define Q4MM_MX_MAX_HEADS 65536
int rope_rotate(const void *x, long long x_token_stride, long long x_head_stride, int dtype, const void *positions,
                int positions_64, const double *frequencies, int rotated, int interleaved, float magnitude, void *out,
                long long out_token_stride, long long out_head_stride, int tokens, int heads, int headDim,
                q4mm_stream_t stream);

/*
 * The paged MX cache.  Keys and values of each of kvHeads heads, headDim
 * values (32, 64, 96 or 128) a token, quantised as by mx_quantize in blocks of
 * 32 along the head, in `pages` pages of pageTokens tokens (a multiple of 16):
 *   codes : [pages][kvHeads][pageTokens] rows of headDim·bits/8 bytes
 *           (16-byte aligned base);
 *   scales: [pages][kvHeads][pageTokens][4] bytes, block b of the head in byte
 *           b, bytes past headDim / 32 written as zero and not read (16-byte
 *           aligned base).
 * k and v each have codes and scales.
 *
 * A batch: sequence i of `sequences` has the rows starts[i] .. starts[i + 1]
 * of a call's dense tensors (starts has sequences + 1 ascending entries), the
 * last of the lengths[i] tokens that it has in the cache with them; its
 * position p lies at place p % pageTokens of page table[i·tableWidth +
 * p / pageTokens].  The three arrays are device memory, 32-bit; a call reads
 * them on its stream, so a captured one may be replayed on new contents.  A
 * page number outside 0 .. pages − 1, or a position beyond the table, is not
 * accessed: q4mm_device_status then reports Q4MM_ERR_INDEX, and what that call
 * computes for the sequence is undefined.  Rows before position 0 (more rows
 * than lengths[i]) are neither written nor read (in mx_attention they see
 * nothing where causal, else what the sequence's other rows see); rows behind the last
 * sequence are left as they were.
 *
 * mx_cache_write — k, v [tokens][kvHeads][headDim] of type dtype, strided as
 * for rope_rotate, to their places: k turned as by rope_rotate at its positions
 * (rotated = 0: as it is) in fp32, near a border between two codes or scales in 64 bits,
 * and then quantised, with no rounding between.
 * Two rows must not have the same place (pages of one table shared with
 * another sequence hold what neither writes).
 *
 * mx_cache_read — the values of the batch's rows, as mx_dequantize gives them.
 *
 * Limits: headDim 32, 64, 96 or 128; bits 4 or 8; pages >= 1;
 *         1 <= kvHeads <= Q4MM_MX_MAX_HEADS; pageTokens a positive multiple of
 *         16, at most 2^24; 0 <= sequences <= 2^24; tableWidth >= 0; tokens and
 *         rotated as for rope_rotate.  No tokens or no sequences: nothing to do.
 * Return Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int mx_cache_write(const void *k, long long k_token_stride, long long k_head_stride, const void *v,
                   long long v_token_stride, long long v_head_stride, int dtype, const double *frequencies,
                   int rotated, int interleaved, float magnitude, void *k_codes, void *k_scales, void *v_codes,
                   void *v_scales, int pages, int kvHeads, int pageTokens, int headDim, int bits, const int *starts,
                   const int *lengths, const int *table, int sequences, int tableWidth, int tokens,
                   q4mm_stream_t stream);
int mx_cache_read(const void *k_codes, const void *k_scales, const void *v_codes, const void *v_scales, int pages,
                  int kvHeads, int pageTokens, int headDim, int bits, const int *starts, const int *lengths,
                  const int *table, int sequences, int tableWidth, void *k, long long k_token_stride,
                  long long k_head_stride, void *v, long long v_token_stride, long long v_head_stride, int dtype,
                  int tokens, q4mm_stream_t stream);

/*
 * mx_attention — attention of a batch's rows over the cache:
 *   y[t][h] = Σ_j softmax_j(scale · q[t][h]·k[j][h / G]) v[j][h / G],
 * G = heads / kvHeads, over the sequence's cached positions j: those up to the
 * row's own where causal, else all lengths[i].  A row that sees none gives
 * zeros.  What a row does not see has no part in it, NaN and infinities
 * included; a block of k that is NaN makes the rows that see it NaN, a block
 * of v those rows' 32 values, and so do codes that are NaN (which no call here
 * writes), those of v their one value.
 * q, y: [tokens][heads][headDim] of type dtype, strided as for rope_rotate,
 * aligned to their elements, not overlapping each other or the cache.
 * Precision: keys and values exact, but that a block whose scale is 2^-17 of
 *         its token's and head's largest counts as zero (of v, that is 32
 *         values of what the token adds to the output); queries exact to
 *         2^-22 of a row's largest value; scores, their maximum, sums and
 *         outputs in fp32 (tensor-core sums lose at most a third of half a step
 *         of dtype with their length).  Probabilities enter the product with
 *         v rounded to 2^-11 of their value, 2^-22 where dtype is Q4MM_F32, or
 *         2^-30 of the row's largest product of a probability and a |v|; before
 *         that their exponents round as fp32 numbers of the size of the score
 *         and of log2 |v|.  With Q4MM_F16 the first of these adds a fifth to a
 *         third to the error that the output's own rounding has.
 *         Rows beside a token whose largest scale byte of v is above 160 or
 *         from 1 to 79 (values of 2^42 and more or below 2^-39, in 4 bits 2^36
 *         and 2^-45), or with NaN among its codes of v, are right too, but take
 *         tens (single tokens) to hundreds (prompts) of times as long.
 *         The same call gives the same bits again.
 * workspace: device memory (16-byte aligned, overlapping nothing else) for the
 *         call to write to, workspace_bytes long; NULL with 0 and any length
 *         are accepted: with less than mx_attention_workspace says the call
 *         may be slower.  Calls that may overlap in time need one each.
 * Limits: as mx_cache_write; heads a multiple of kvHeads; tokens · G at most
 *         Q4MM_MX_MAX_ROWS; scale finite, >= 0.  Positions from 2^31 - 256 on
 *         are beyond any table.
 * Returns Q4MM_OK or Q4MM_ERR_{DIM,NULL,ALIGN,ALIAS,CUDA}.
 */
int mx_attention(const void *q, long long q_token_stride, long long q_head_stride, int dtype, const void *k_codes,
                 const void *k_scales, const void *v_codes, const void *v_scales, int pages, int kvHeads,
                 int pageTokens, int headDim, int bits, const int *starts, const int *lengths, const int *table,
                 int sequences, int tableWidth, float scale, int causal, void *y, long long y_token_stride,
                 long long y_head_stride, int tokens, int heads, void *workspace, size_t workspace_bytes,
                 q4mm_stream_t stream);

/*
 * mx_attention_workspace — bytes of workspace with which mx_attention, on the
 * current device, uses every SM for a call of these sizes: more than none where
 * few rows meet a long cache.  0 also for sizes that mx_attention refuses.
 */
size_t mx_attention_workspace(int kvHeads, int pageTokens, int headDim, int sequences, int tableWidth, int tokens,
                              int heads);

/*
 * q4mm_call — one of the calls named below with its arguments, in their order,
 * in 8-byte words: pointers, strides and sizes as they are, integers sign-
 * extended, a float as a double.  For bindings that pay for every argument of
 * a foreign call.  Returns what the call returns.
 */
enum { Q4MM_CALL_ROPE_ROTATE = 0, Q4MM_CALL_MX_CACHE_WRITE = 1, Q4MM_CALL_MX_CACHE_READ = 2, Q4MM_CALL_MX_ATTENTION = 3 };
int q4mm_call(int which, const long long *words);

/* Message for the last error returned on the calling thread ("" if none).
 * The pointer stays valid until the thread's next failing call. */
const char *q4mm_last_error(void);

/*
 * q4mm_device_status — waits for `stream`, then returns Q4MM_OK, or
 * Q4MM_ERR_TIMEOUT if a bounded in-kernel wait of an earlier call on the
 * current device ran out, or Q4MM_ERR_INDEX if one met a page number or a
 * position outside its cache or table.  clear != 0 resets the status word afterwards.
 * Returns Q4MM_ERR_CUDA if the stream reports an error.
 */
int q4mm_device_status(q4mm_stream_t stream, int clear);

/*
 * q4mm_test_fail_next_wait — a test hook for the library's failure
 * detection; the pages have no counterpart.  The calling thread's next call
 * of q4k_matmul (one-token and 3-8 token kernels), q4_0_gemv, q6k_gemv,
 * q4k_ffn_swiglu, q4k_matmul_tc, mx_matmul or mx_attention (many rows) never
 * issues the copy of weight stage `stage` of each CTA (its ring stage, its
 * 256-row weight tile on the tensor cores, or its tile of 128 keys, the last
 * if it has fewer) and bounds every in-kernel wait by `limit_cycles` SM cycles
 * (about 2·10^6 per millisecond) instead of about 2·10^9.  The waits on the
 * missing stage then run out: the kernel sets the device status word, lets
 * every copy it did issue land, and exits; that call's y is undefined and
 * q4mm_device_status reports Q4MM_ERR_TIMEOUT.  Nothing faults or waits
 * without a bound.  Later calls, and calls on other threads, are not
 * affected; a call rejected by validation leaves it armed.  stage = -1
 * disarms it; otherwise stage >= 0 and limit_cycles > 0, else Q4MM_ERR_DIM.
 */
int q4mm_test_fail_next_wait(int stage, long long limit_cycles);

/*
 * q4mm_test_attention_kernel — a test hook: the calling thread's mx_attention
 * (and mx_attention_workspace) take the kernel for few rows (1) or the one for
 * many (2) whatever the sizes, until 0 leaves the choice to the library again.
 * Else Q4MM_ERR_DIM.
 */
int q4mm_test_attention_kernel(int which);

/* Library version, major·10000 + minor·100 + patch. */
int q4mm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* Q4MM_H */

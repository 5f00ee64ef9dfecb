/*
 * nvfp4.h -- C ABI of libnvfp4.so: the NVFP4 (E2M1 codes + E4M3 scale per 16
 * elements + FP32 per-tensor scale) W4A4 linear and MLP hot path on one
 * Blackwell GPU (sm_103a).
 *
 * Sources, by page title and section:
 *  - "PERFORMANCE -- verified hot-path audit and prioritized fixes"
 *    (nvfp4-megamoe-kernel PERFORMANCE_AUDIT.md): P0 (activation global
 *    scale amax/(6*448) computed on the device and handed to the kernel as a
 *    (1,) device tensor, never read back by the host), P8 items 1-2
 *    (quantization fused into the producer: RMSNorm + quantize), DOCTRINE 1
 *    (no host state on the hot path).
 *  - "CUDA: NVFP4 prefill on Blackwell leaves ~1.45x performance on the
 *    table. Comparison + PoC" (llama.cpp discussion 28514), "What the patch
 *    does": GLU output quantized straight into the next GEMM's activation
 *    format, gate/up sharing one quantized input, batched-row rms_norm,
 *    TMA + mbarrier fed FP4 MMA tiles; and its ncu finding that a 36-byte
 *    interleaved FP4 block is only 4-byte aligned -- codes and scales are
 *    therefore kept in separate, 16-byte aligned arrays here.
 *  - "tp>1 prefill is host-bound: per-token fp4 GEMM + per-layer H2D
 *    activation staging" (vllm.cpp issue 2144), "Fix directions" 1-3: one
 *    launch set per T-token batch with a grid that scales with T,
 *    activations resident on the device, quantization on the device.
 *
 * Conventions (all functions):
 *  - Every pointer argument is a DEVICE pointer unless stated otherwise, owned
 *    by the caller.  No function allocates, frees or synchronises; all work is
 *    enqueued on `stream` (a cudaStream_t; NULL is the legacy default stream).
 *  - The GEMM kernels use programmatic dependent launch: they may start
 *    while the previous kernel of the stream still runs, and read their
 *    operands only after it has completed -- except inside nvfp4_mlp, whose
 *    GEMMs fetch the weights early (the weights were complete before the
 *    call's first, plainly launched kernel started): a tensor quantized by
 *    the launch just before a GEMM call is safe to use as its weight.
 *  - The return value is a status (NVFP4_OK = 0).  Argument errors are
 *    detected on the host before anything is enqueued.  NVFP4_ERR_CUDA
 *    reports a launch error (cudaGetLastError); asynchronous failures show
 *    up in the stream as usual.
 *  - bf16 tensors are row-major with a row pitch given in ELEMENTS; bf16
 *    base pointers and pitches must be 16-byte aligned (pitch % 8 == 0).
 *  - A quantized tensor (nvfp4_tensor_t) of logical shape [rows x cols]:
 *      codes: byte (r, k/2) at codes + r*ld + k/2 holds element k in its low
 *             nibble when k is even, in its high nibble when k is odd; each
 *             nibble is an E2M1 code (bit 3 sign, magnitudes 0, .5, 1, 1.5,
 *             2, 3, 4, 6).  cols % 64 == 0; ld % 16 == 0; codes 16-B aligned.
 *      sf:    one unsigned E4M3 scale per 16 consecutive elements of a row,
 *             in 512-byte tiles of 128 rows x 4 scales: rows padded to a
 *             multiple of 128, scale columns (cols/16) padded to a multiple of
 *             4, tiles row-tile-major, and inside a tile the scale of row r,
 *             column c at (r%32)*16 + (r%128)/32*4 + c%4.  Size:
 *             nvfp4_sf_bytes(rows, cols); 128-B aligned; padding bytes are 0.
 *      g:     fp32[1] per-tensor global scale (> 0).
 *    Element value = E2M1(code) * E4M3(scale) * g.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* nvfp4_stream_t; /* identical to cudaStream_t */

enum nvfp4_status {
    NVFP4_OK = 0,
    NVFP4_ERR_INVALID_ARG = 1, /* NULL pointer, bad shape (rows < 1, cols % 64 != 0, ...) */
    NVFP4_ERR_MISALIGNED = 2,  /* pointer or pitch not aligned as documented */
    NVFP4_ERR_UNSUPPORTED = 3, /* device is not compute capability 10.3 (sm_103a) */
    NVFP4_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed */
    NVFP4_ERR_WORKSPACE = 5,   /* workspace missing or smaller than required */
    NVFP4_ERR_TIMEOUT = 6      /* device-side: a pipeline wait exceeded its time limit */
};

/* Intermediate (SwiGLU output) global-scale modes of the fused gate/up GEMM. */
enum nvfp4_inter_mode {
    /* g_inter is an input: a scale fixed ahead of time (e.g. by one DYNAMIC
     * warm-up call), used by the GEMM epilogue to requantize SwiGLU output
     * straight into FP4 ("keep the warm-up scale as a device tensor"). */
    NVFP4_INTER_STATIC = 0,
    /* g_inter is an output: the epilogue stores bf16 SwiGLU output and its
     * amax, then the scale max(amax,1e-8)/2688 is written to *g_inter on the
     * device and the SwiGLU output is quantized with it (exact per-call
     * scale, two extra HBM passes over T x I bf16). */
    NVFP4_INTER_DYNAMIC = 1
};

/* A quantized matrix; see the conventions above. */
typedef struct {
    const uint8_t* codes;
    const uint8_t* sf;
    const float* g;
    int64_t rows;
    int64_t cols;
    int64_t ld; /* bytes */
} nvfp4_tensor_t;

/* ------------------------------------------------------------ host helpers */

/* Bytes of a codes array with ld = cols/2: rows * cols / 2. */
size_t nvfp4_codes_bytes(int64_t rows, int64_t cols);
/* Bytes of a scale array: pad128(rows) * pad4(cols/16). */
size_t nvfp4_sf_bytes(int64_t rows, int64_t cols);
/* Workspace of nvfp4_amax_scale and nvfp4_scale_quantize (256 bytes, 256-B aligned). */
size_t nvfp4_amax_workspace_bytes(void);
/* Workspace that lets nvfp4_gemm split its work evenly over all SMs of the
 * current device (8 KB of ready flags + 128 KB per SM; 0 when no device is
 * usable). */
size_t nvfp4_gemm_workspace_bytes(void);
/* Workspace of nvfp4_gemm_swiglu for an A of T rows and an intermediate of I
 * columns on the current device: 256 + 8192 bytes, + T*I*2 (DYNAMIC), + the
 * split schedule's 128 KB per SM.  A workspace without the last part is
 * accepted (the call then runs unsplit). */
size_t nvfp4_swiglu_workspace_bytes(int64_t T, int64_t I, int inter_mode);
/* Workspace of nvfp4_mlp (T tokens, hidden H, intermediate I) on the current
 * device; likewise, its last 128 KB per SM (the split schedule's) may be
 * left out. */
size_t nvfp4_mlp_workspace_bytes(int64_t T, int64_t H, int64_t I, int inter_mode);
/* Workspace of nvfp4_gemm_experts for T tokens, topk slots, K columns and E
 * experts: the routing tables plus the expert-sorted operand (at most
 * T*topk + 127*min(E, T*topk) rows, rounded up to 128, of K/2 + K/16 bytes). */
size_t nvfp4_experts_workspace_bytes(int64_t T, int64_t topk, int64_t K, int64_t num_experts);
/* Static description of a status code. */
const char* nvfp4_status_string(int status);
/* Reads (and if clear != 0 resets) the library's device-side status word of
 * the current device, which kernels set when a pipeline wait times out.
 * SYNCHRONOUS (a device-to-host copy); diagnostics and tests only. */
int nvfp4_device_status(int* status_out, int clear);
/* Measures the issue rate of the tensor-core instruction form the GEMM
 * kernels use (tcgen05.mma.cta_group::2 kind::mxf4nvf4 scale_vec::4X,
 * M=256 N=256 K=64, with its scale copies), fed back to back from operands
 * already in shared memory on one SM pair of the current device: writes
 * the multiply-adds per SM per clock cycle to *mac_per_clk.  Returns
 * NVFP4_ERR_TIMEOUT if the measurement's bounded wait ran out.  SYNCHRONOUS;
 * a measurement diagnostic (the dense NVFP4 peak of this instruction is
 * 2 * mac_per_clk * SMs * SM clock), not part of the path.  No counterpart
 * in the pages, which give no peak. */
int nvfp4_mma_issue_rate(double* mac_per_clk);

/* ------------------------------------------------------------- the path */

/*
 * nvfp4_amax_scale -- device per-tensor global scale.
 *   g_out[0] = max(amax, 1e-8) / (6 * 448)  (binary32 division),
 *   amax = max |v| over the bf16 matrix v.
 * Source: "PERFORMANCE -- verified hot-path audit and prioritized fixes", P0
 * (the runtime scale, computed on the device instead of via .item()).
 *   x        bf16 [rows x cols], row pitch ldx elements.
 *   norm_w   NULL, or bf16 [cols]: then v is the RMSNorm of x,
 *            v = bf16(x * r * w), r = 1/sqrt(mean(x^2) + eps) per row
 *            (the batched-row RMSNorm prologue).
 *   g_out    fp32[1], written.
 *   workspace >= nvfp4_amax_workspace_bytes(), 256-B aligned.  It must be
 *            zero-filled ONCE after allocation; every call returns it to zero.
 *            Calls sharing one workspace must be stream-ordered.
 * Requires rows >= 1, cols >= 8, cols % 8 == 0.
 */
int nvfp4_amax_scale(const void* x, int64_t rows, int64_t cols, int64_t ldx,
                     const void* norm_w, float eps, float* g_out,
                     void* workspace, size_t workspace_bytes, nvfp4_stream_t stream);

/*
 * nvfp4_quantize -- bf16 -> NVFP4 with the device global scale g.
 * Per 16-element block (binary32, one rounding per step):
 *   s = E4M3_rne_satfinite( amax16 / (6*g) ),
 *   code_i = s == 0 ? +0 : E2M1_rne_satfinite( v_i / (E4M3(s) * g) ).
 * Sources: "PERFORMANCE -- verified hot-path audit and prioritized fixes",
 * P0 and P8 item 2 (rmsnorm_quantize); "CUDA: NVFP4 prefill on Blackwell
 * leaves ~1.45x performance on the table", item 2 (batched-row rms_norm).
 *   x, ldx, norm_w, eps  as nvfp4_amax_scale (norm_w != NULL: quantize the
 *            RMSNorm of x, computed exactly as nvfp4_amax_scale computes it).
 *   g        fp32[1] device global scale.
 *   codes    [rows][ld_codes] bytes, ld_codes >= cols/2, % 16 == 0.
 *   sf       nvfp4_sf_bytes(rows, cols) bytes, 128-B aligned; padding written 0.
 *   y_out    NULL, or bf16 [rows x cols] (pitch cols): receives v (export for
 *            tests of the norm prologue).
 * Requires rows >= 1, cols % 64 == 0.
 */
int nvfp4_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx,
                   const void* norm_w, float eps, const float* g,
                   uint8_t* codes, int64_t ld_codes, uint8_t* sf, void* y_out,
                   nvfp4_stream_t stream);

/*
 * nvfp4_scale_quantize -- nvfp4_amax_scale then nvfp4_quantize with the
 * scale just computed, as ONE kernel launch: *g_out, codes and sf are bit for
 * bit those of the two calls.  The kernel is a cooperative launch with one
 * grid-wide barrier between the amax and the quantization (every block is
 * resident; when the grid covers all rows at once each row is read once).
 * Sources: as nvfp4_amax_scale and nvfp4_quantize.
 *   x, ldx, norm_w, eps  as nvfp4_amax_scale.
 *   g_out    fp32[1], written with the global scale.
 *   codes, ld_codes, sf  as nvfp4_quantize.
 *   workspace as nvfp4_amax_scale (>= nvfp4_amax_workspace_bytes(), zero-filled
 *            once; calls leave it zeroed).  After a call that reported a
 *            timeout through nvfp4_device_status it must be zero-filled again.
 * Requires rows >= 1, cols % 64 == 0.
 */
int nvfp4_scale_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx,
                         const void* norm_w, float eps, float* g_out,
                         uint8_t* codes, int64_t ld_codes, uint8_t* sf,
                         void* workspace, size_t workspace_bytes, nvfp4_stream_t stream);

/*
 * nvfp4_gemm -- block-scaled GEMM on the tensor cores (tcgen05
 * kind::mxf4nvf4, fp32 accumulation in tensor memory):
 *   out[m][n] = bf16( alpha * sum_k A[m,k] W[n,k] ),  alpha = fp32(gA * gW),
 *   or, with residual != NULL, bf16( residual[m][n] + that bf16 ).
 * Source: "CUDA: NVFP4 prefill on Blackwell leaves ~1.45x performance on the
 * table" item 3 (TMA + mbarrier fed FP4 MMA accumulated in place);
 * "tp>1 prefill is host-bound" fix direction 1 (one launch for all T rows).
 *   A        activations, rows M = T (any M >= 1), cols K.
 *   W        weights [N x K] (K-major, as nn.Linear stores them).
 *   out      bf16 [M x N], pitch ldo; may alias residual (same pitch).
 *   workspace NULL, or >= 8192 bytes, 256-B aligned, zero-filled once after
 *            allocation (calls leave it zeroed); calls sharing one workspace
 *            must be stream-ordered.  With nvfp4_gemm_workspace_bytes() bytes
 *            the GEMM may split its tiles' K ranges over all SMs when whole
 *            tiles would leave part of the GPU idle (fp32 partials combined
 *            in the workspace); otherwise whole tiles are spread over the SMs.
 * With M <= 8 and such a workspace the GEMM runs instead as a weight stream
 * on the tensor cores (the weights as the MMA's 128-row side, split over
 * all SMs along K, fp32 partials combined in the workspace in a fixed
 * order); without one, with M <= 2 and at most 32 MiB of weight codes, as
 * a weight stream on the CUDA cores (exact int32 sums of E2M1 code
 * products per 16-element block, block scales applied exactly in fp32,
 * fp32 accumulation).  Either gives the same result up to the fp32
 * summation order.  nvfp4_gemm_swiglu and nvfp4_mlp do the same, except
 * that a SwiGLU GEMM whose 128-column blocks fill at least 85% of the SMs
 * runs as whole tiles.
 * Requires K == A->cols == W->cols, K % 64 == 0, N % 16 == 0.
 */
int nvfp4_gemm(const nvfp4_tensor_t* A, const nvfp4_tensor_t* W,
               void* out, int64_t ldo, const void* residual, int64_t ldr,
               void* workspace, size_t workspace_bytes, nvfp4_stream_t stream);

/* Rotary embedding applied by nvfp4_gemm_rope (all pointers DEVICE). */
typedef struct {
    const int32_t* pos;   /* int32 [M]: position of each output row, in [0, positions) (below) */
    const float* cos_t;   /* fp32 [positions x table_ld]: cos of the angle of (position, pair i) at [p*table_ld + i] */
    const float* sin_t;   /* fp32, the same layout: sin of that angle */
    int64_t table_ld;     /* floats per table row, >= rope_dim / 2 */
    int64_t positions;    /* rows of the tables, >= 1 */
    int64_t col0;         /* first output column of the first rotated head; even */
    int64_t heads;        /* rotated heads (col0 + heads * head_dim <= N) */
    int64_t head_dim;     /* columns per head; even */
    int64_t rope_dim;     /* rotated columns per head: the LAST rope_dim of each head; even, <= head_dim */
    int inverse;          /* nonzero: the inverse rotation */
} nvfp4_rope_t;

/*
 * nvfp4_gemm_rope -- nvfp4_gemm (no residual) with a rotary position
 * embedding applied to its bf16 output in the GEMM's epilogue, e.g. the Q
 * and K heads of a QKV projection.  Source: "PERFORMANCE -- verified
 * hot-path audit and prioritized fixes", P5 (RoPE on the last rope_dim
 * columns of each head, float32 arithmetic from bf16 and back) and the
 * structural target "fuse RoPE into the Q/KV GEMM epilogue".
 * In a rotated head, the pairs (e, o) = (y[2i], y[2i+1]) of the last rope_dim
 * columns of y = nvfp4_gemm's bf16 output are rotated with
 * c = cos_t[pos[m]*table_ld + i], s = sin_t[...]:
 *   forward: e' = e*c - o*s,  o' = e*s + o*c;  inverse: e' = e*c + o*s,  o' = o*c - e*s
 * each product, sum and difference one binary32 operation, then rounded to
 * bf16; every other column is nvfp4_gemm's output.  A position outside the
 * tables takes their first or last row, whichever is nearer, and records
 * NVFP4_ERR_INVALID_ARG * 100 + 33 in the device status word.
 *   A, W, out, ldo, workspace  as nvfp4_gemm.
 *   rope     the embedding's tables and geometry (above).
 */
int nvfp4_gemm_rope(const nvfp4_tensor_t* A, const nvfp4_tensor_t* W, void* out, int64_t ldo,
                    const nvfp4_rope_t* rope, void* workspace, size_t workspace_bytes,
                    nvfp4_stream_t stream);

/*
 * nvfp4_gemm_experts -- expert-indexed GEMM, the routed projection of a
 * mixture-of-experts layer (llama.cpp's MUL_MAT_ID).  For token t and routing
 * slot j < topk, with e = ids[t*topk + j]:
 *   out[(t*topk + j) * ldo + n] = bf16( fp32(A->g[0] * W->g[e]) * sum_k A[t,k] W_e[n,k] ),
 * the sum and the rounding as in nvfp4_gemm.  The routing table stays on
 * the device: three launches (routing, gather of the routed rows into an
 * expert-sorted operand, grouped tcgen05 GEMM over a tile table built on the
 * device), no host synchronisation.  Sources: "CUDA: NVFP4 prefill on
 * Blackwell leaves ~1.45x performance on the table" (the MUL_MAT_ID tests
 * its patch passes); "PERFORMANCE -- verified hot-path audit and prioritized
 * fixes" (the routed experts run without a host read of the routing table).
 *   A            [T x K] quantized activations.
 *   W            the E experts' weights stacked: rows E*N (expert e = rows
 *                e*N .. e*N + N - 1), cols K; W->g points to fp32[E], expert
 *                e's global scale.  N = W->rows / E, a multiple of 128.
 *   num_experts  E, 1 .. 4096.
 *   ids          DEVICE int32 [T * topk]: the expert of each (token, slot).
 *                An id outside [0, E) leaves that output row unwritten and
 *                records NVFP4_ERR_INVALID_ARG * 100 + 30 in the device
 *                status word (nvfp4_device_status).
 *   topk         routing slots per token, >= 1 (T * topk < 2^31).
 *   out          bf16 [T*topk x N], row pitch ldo (elements).
 *   workspace    nvfp4_experts_workspace_bytes(T, topk, K, E) bytes,
 *                256-byte aligned; no zero-fill needed; not shared with a
 *                call that may run at the same time.
 */
int nvfp4_gemm_experts(const nvfp4_tensor_t* A, const nvfp4_tensor_t* W, int64_t num_experts, const int32_t* ids,
                       int64_t topk, void* out, int64_t ldo, void* workspace, size_t workspace_bytes,
                       nvfp4_stream_t stream);

/*
 * nvfp4_gemm_swiglu -- fused gate/up GEMM with SwiGLU epilogue and FP4
 * requantization into the down projection's activation format:
 *   gate = bf16(alpha_g * A Wg^T), up = bf16(alpha_u * A Wu^T),
 *   s = bf16( gate * sigmoid(gate) * up ),  S = NVFP4(s) with scale g_inter.
 * Source: "CUDA: NVFP4 prefill on Blackwell leaves ~1.45x performance on the
 * table" item 2 (GLU output quantized directly into the next GEMM's
 * activation format; gate and up share one quantized input).
 *   A            [T x K] quantized input, shared by both GEMMs.
 *   W_gate, W_up [I x K] each, same shape.
 *   inter_mode   NVFP4_INTER_STATIC (g_inter read) or NVFP4_INTER_DYNAMIC
 *                (g_inter written with the per-call scale).
 *   s_codes      [T][ld_s_codes] bytes (I/2 per row); s_sf nvfp4_sf_bytes(T, I).
 *   s_bf16       NULL, or bf16 [T x I] (pitch I): receives s (export).
 *   workspace    nvfp4_swiglu_workspace_bytes(T, I, inter_mode), 256-B aligned,
 *                zero-filled once after allocation (calls leave it zeroed).
 * Requires I % 128 == 0, K % 64 == 0.
 */
int nvfp4_gemm_swiglu(const nvfp4_tensor_t* A, const nvfp4_tensor_t* W_gate,
                      const nvfp4_tensor_t* W_up, int inter_mode, float* g_inter,
                      uint8_t* s_codes, int64_t ld_s_codes, uint8_t* s_sf, void* s_bf16,
                      void* workspace, size_t workspace_bytes, nvfp4_stream_t stream);

/*
 * nvfp4_mlp -- the whole NVFP4 MLP block for a batch of T tokens in one
 * launch set, activations device-resident, no host synchronisation:
 *   h   = NVFP4( RMSNorm(x; norm_w, eps) )   (scale g_h computed on device)
 *   S   = nvfp4_gemm_swiglu(h, W_gate, W_up, inter_mode, g_inter)
 *   out = bf16( [x +] alpha_d * S W_down^T )
 * Sources: all three pages (see top of file).
 *   x        bf16 [T x H], pitch ldx.
 *   W_gate, W_up [I x H]; W_down [H x I].
 *   out      bf16 [T x H], pitch ldo; may alias x (in-place residual, ldo == ldx).
 *   workspace nvfp4_mlp_workspace_bytes(T, H, I, inter_mode), 256-B aligned,
 *            zero-filled once after allocation (calls leave it zeroed).
 * Requires H % 64 == 0, I % 128 == 0, T >= 1.
 */
int nvfp4_mlp(const void* x, int64_t T, int64_t H, int64_t ldx,
              const void* norm_w, float eps,
              const nvfp4_tensor_t* W_gate, const nvfp4_tensor_t* W_up,
              const nvfp4_tensor_t* W_down, int inter_mode, float* g_inter,
              void* out, int64_t ldo, int add_residual,
              void* workspace, size_t workspace_bytes, nvfp4_stream_t stream);

/*
 * nvfp4_mlp_noalloc -- nvfp4_mlp for callers that cannot allocate device
 * memory (no counterpart on the source pages; an addition of this library).
 * Examples: a plugin that only receives borrowed tensor pointers from its host
 * application and has no allocator, or a latency-critical caller for which
 * cudaMalloc -- which may synchronise the whole device -- is not acceptable.
 *
 * Same computation, arguments, requirements and results as nvfp4_mlp, minus
 * the workspace: the intermediates live in a fixed 32 MiB array inside this
 * library (every GPU that loads the library holds it until the process
 * exits).  The array must hold nvfp4_mlp's workspace without the split
 * schedule's partial slots (those slots are used too when they also fit,
 * which at H=5120, I=17408 and 152 SMs is up to T ~1070 with
 * NVFP4_INTER_STATIC): a larger call returns NVFP4_ERR_WORKSPACE.  At
 * H=5120, I=17408 the largest T is 2642 with NVFP4_INTER_STATIC and 704 with
 * NVFP4_INTER_DYNAMIC.
 *   - Argument errors (the statuses nvfp4_mlp returns) and
 *     NVFP4_ERR_WORKSPACE are returned before anything is enqueued.
 *   - Allocates nothing and calls no allocator.  It enqueues one small
 *     cudaMemsetAsync that clears the array's amax words and the split
 *     schedule's flag words (a call that stopped early may have left them
 *     non-zero), then the nvfp4_mlp launches.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it for the life of the process; make
 *     that first call before any stream capture.  The cached address is not
 *     looked up again: do not use the library across cudaDeviceReset or
 *     anything else that destroys the device's primary context.
 *   - Every call shares the one array: calls that can overlap on the GPU
 *     (different streams, or several host threads) race with each other and
 *     must be serialised by the caller.
 */
int nvfp4_mlp_noalloc(const void* x, int64_t T, int64_t H, int64_t ldx,
                      const void* norm_w, float eps,
                      const nvfp4_tensor_t* W_gate, const nvfp4_tensor_t* W_up,
                      const nvfp4_tensor_t* W_down, int inter_mode, float* g_inter,
                      void* out, int64_t ldo, int add_residual, nvfp4_stream_t stream);

/*
 * nvfp4_noalloc_scratch -- diagnostics: the device address (on the current
 * device) and the size of nvfp4_mlp_noalloc's fixed array.  The array
 * belongs to nvfp4_mlp_noalloc; a caller may read it, or clear it between
 * calls, but anything it writes there is overwritten or cleared by the next
 * call.  Same caching as nvfp4_mlp_noalloc.
 */
int nvfp4_noalloc_scratch(void** device_ptr, size_t* bytes);

/* ------------------------------------------- attention over a paged KV cache
 *
 * One step of a serving loop gives every request r some new tokens (q_len[r]:
 * 1 when decoding, a chunk of its prompt when prefilling) on top of those
 * already in the cache (ctx_len[r]).  The new tokens of all requests are
 * packed, request after request, into the rows of one matrix.
 *   nvfp4_attn_plan    once per step: packed offsets, positions, block tables,
 *                      slots and the attention's work schedule, from the lengths
 *   nvfp4_kv_append    per layer: the new tokens' K and V rows into the cache
 *   nvfp4_attn_paged   per layer: attention of the new tokens over the cache
 *   nvfp4_attn_prompt  per layer, without a cache: attention within packed prompts
 * The lengths stay on the device: no call reads them on the host, and the
 * calls of a step can be captured in a CUDA graph and replayed with new
 * lengths.  The pages have no attention core (they measure the projections
 * around it); these are additions of this library.
 */

/* The tables of one step (device pointers, int32 arrays unless stated). */
typedef struct {
    int64_t requests;          /* R, 1 .. 8192 */
    int64_t tokens;            /* rows of the packed matrices; >= sum of q_len (rows past it are padding) */
    const int32_t* q_len;      /* [R] new tokens of each request, >= 0 */
    const int32_t* ctx_len;    /* [R] tokens already in the cache, >= 0; NULL: none */
    int32_t* cu_q;             /* [R+1] out: first packed row of each request; cu_q[R] = all new tokens */
    int32_t* kv_len;           /* [R] out: ctx_len + q_len */
    int32_t* pos;              /* [tokens] out: position of each packed row (0 for padding rows), or NULL */
    /* paged cache; page_size 0: none, and the rest of this group is ignored */
    int64_t page_size;         /* tokens per page: 16, 32, 64 or 128 */
    int32_t* block_table;      /* [R x table_cols], row pitch table_ld: page of tokens j*page_size .. of request r */
    int64_t table_cols, table_ld;
    int32_t* slot;             /* [tokens] out: page * page_size + row of each packed row; -1: none */
    const int32_t* free_pages; /* [free_count] free page ids, taken in order; NULL: block_table is complete already */
    int64_t free_count;
    const int32_t* cursor;     /* [1] entries of free_pages already taken, or NULL: 0 */
    int32_t* cursor_out;       /* [1] out: cursor + pages taken by this step (may alias cursor), or NULL */
    /* attention; heads 0: no schedule */
    int64_t heads, kv_heads;   /* heads % kv_heads == 0, heads / kv_heads <= 128 */
    int64_t window;            /* keys a row sees, its own included; 0: all up to its own */
    void* schedule;            /* nvfp4_attn_schedule_bytes() bytes, 256-B aligned, out */
    size_t schedule_bytes;
} nvfp4_step_t;

/* A paged KV cache: page p, kv head h, row i, column d of K at
 * k + p*page_stride + (h*page_size + i)*head_dim + d (elements); V likewise. */
typedef struct {
    void* k;                   /* bf16 */
    void* v;                   /* bf16 */
    int64_t pages, page_size, kv_heads, head_dim;
    int64_t page_stride;       /* elements, >= kv_heads*page_size*head_dim, % 8 == 0 */
} nvfp4_kv_cache_t;

/* Query rows, outputs and scaling of one attention call: the row of token t,
 * head h starts at q + t*ldq + h*hq (elements), its output at out + t*ldo + h*ho. */
typedef struct {
    const void* q;             /* bf16 [tokens][heads][head_dim] */
    int64_t ldq, hq;
    void* out;                 /* bf16 [tokens][heads][head_dim] */
    int64_t ldo, ho;
    float* lse;                /* NULL, or fp32 [tokens x heads]: log of the row's sum of exp(score) */
    int64_t head_dim;          /* 16 .. 128, % 8 == 0 */
    float scale;               /* score = scale * q.k; finite, at most FLT_MAX / 1.5 */
    int32_t zero_padding;      /* rows of padding (cu_q[R] .. tokens - 1): 0 not written; else out 0, lse -inf */
} nvfp4_attn_io_t;

/* Bytes of a step's schedule for any lengths of R requests and tokens rows. */
size_t nvfp4_attn_schedule_bytes(int64_t requests, int64_t tokens, int64_t heads, int64_t kv_heads);
/* Workspace of the attention calls on the current device, any sizes. */
size_t nvfp4_attn_workspace_bytes(void);

/*
 * nvfp4_attn_plan -- the tables of a step from its requests' lengths, in one
 * launch (two where cursor_out is cursor).  With need(x) = ceil(x / page_size) pages for x tokens:
 *   cu_q[r+1] = cu_q[r] + q_len[r],  kv_len[r] = ctx_len[r] + q_len[r];
 *   packed row cu_q[r] + t: pos = ctx_len[r] + t,
 *                           slot = block_table[r][pos / page_size] * page_size + pos % page_size;
 *   request r takes need(kv_len[r]) - need(ctx_len[r]) pages from free_pages,
 *   request after request from *cursor on, into block_table[r][need(ctx_len[r])] ...
 *   (earlier entries are read, never written).
 * Rows past the last token get pos 0 and slot -1.  A negative length counts as
 * 0; tokens past `tokens` are dropped; a row whose page does not exist (the
 * free list ran out, the table has no such column) gets slot -1, its table
 * entry -1.  A schedule of more than 2^30 units (2 + ceil(keys / 128) for each
 * kv head of each tile of rows) ends with the last whole item before that; the
 * rows behind get no attention, nor do rows at positions from 2^30 on a right
 * one.  Each of these records
 * NVFP4_ERR_INVALID_ARG * 100 + 31 in the device status word.  *cursor_out counts the pages asked for, so that a value
 * above free_count tells how many were missing.  q_len and ctx_len are none of
 * the outputs (a loop keeps its own ctx_len beside kv_len).
 */
int nvfp4_attn_plan(const nvfp4_step_t* step, nvfp4_stream_t stream);

/*
 * nvfp4_kv_append -- writes packed row t of K and V, all kv heads, into slot
 * slot[t] of the cache (bf16 copied bit for bit):
 *   k_cache[slot / page_size][h][slot % page_size][:] = k[t][h][:];  v likewise.
 *   k, v     bf16, row of token t, head h at k + t*ldk + h*hk (elements);
 *            16-byte aligned, pitches % 8 == 0.
 *   slot     int32 [tokens]; -1 is skipped; any other value outside the cache
 *            is skipped and records NVFP4_ERR_INVALID_ARG * 100 + 32.  No slot
 *            appears twice.
 *   cache    its page_size is the one of the step that made the slots (which a
 *            slot does not tell).
 */
int nvfp4_kv_append(const void* k, int64_t ldk, int64_t hk, const void* v, int64_t ldv, int64_t hv,
                    const int32_t* slot, int64_t tokens, const nvfp4_kv_cache_t* cache, nvfp4_stream_t stream);

/*
 * nvfp4_attn_prompt -- causal attention within packed prompts (the rows of
 * request r are cu_q[r] .. cu_q[r+1] - 1 of q, k and v alike), grouped heads:
 *   head h reads kv head h / (heads / kv_heads);
 *   row t of a request sees keys max(0, t - window + 1) .. t of that request;
 *   out = bf16( sum_j softmax_j(scale * q.k_j) v_j ),  lse = log sum_j exp(scale * q.k_j).
 * Scores, softmax statistics and sums are binary32; the probabilities are
 * rounded to bf16 for the product with V.  Rows past cu_q[R] as io->zero_padding says.
 * A value that is not finite can make rows of its own request NaN that do not
 * see its key (0 * NaN), never another request's.
 *   step     after nvfp4_attn_plan on the same stream order, with a schedule
 *            and ctx_len NULL.  A step with pages serves too (its slots take the
 *            same prompts into the cache), as far as its block table reaches:
 *            a request's keys from table_cols * page_size on, which the plan
 *            reports, are seen by no row.
 *   k, v     as nvfp4_kv_append.
 *   workspace nvfp4_attn_workspace_bytes() bytes, 256-B aligned, zero-filled
 *            once after allocation (calls leave its counters zeroed; after a
 *            reported timeout zero it again); calls sharing it must be
 *            stream-ordered.
 */
int nvfp4_attn_prompt(const nvfp4_step_t* step, const nvfp4_attn_io_t* io, const void* k, int64_t ldk, int64_t hk,
                      const void* v, int64_t ldv, int64_t hv, void* workspace, size_t workspace_bytes,
                      nvfp4_stream_t stream);

/*
 * nvfp4_attn_paged -- attention of a step's new tokens over the paged cache,
 * which holds their own K and V already (nvfp4_kv_append): row t of request r
 * is at position p = kv_len[r] - q_len[r] + t and sees cache positions
 * max(0, p - window + 1) .. p of its request, found through block_table.  The
 * rest as nvfp4_attn_prompt.  Cache rows that no row of the request sees may
 * hold anything, NaN included.  A row that sees no key (its window lies past the table's last
 * column) gives out 0 and lse -inf.  A page id outside the cache counts as a page of zeros.
 */
int nvfp4_attn_paged(const nvfp4_step_t* step, const nvfp4_attn_io_t* io, const nvfp4_kv_cache_t* cache,
                     void* workspace, size_t workspace_bytes, nvfp4_stream_t stream);

/* -------------------------------------------- norms and rotation of heads
 *
 * What lies between a QKV projection and the attention where the model
 * normalises its query and key heads.
 */

typedef struct nvfp4_kv4_cache nvfp4_kv4_cache_t;   /* below */

/* Heads of one call: the row of token t, head h of a matrix x starts at
 * x + t*ldx + h*hx (elements), 16-byte aligned, pitches % 8 == 0. */
typedef struct {
    int64_t tokens;            /* >= 1 */
    int64_t heads, kv_heads;   /* of q and of k and v; one of them may be 0 */
    int64_t head_dim;          /* 16 .. 128, % 8 == 0 */
    const void* q;             /* bf16 [tokens][heads][head_dim] */
    int64_t ldq, hq;
    void* q_out;               /* likewise; may be q with its pitches */
    int64_t ldqo, hqo;
    const void* k;             /* bf16 [tokens][kv_heads][head_dim] */
    int64_t ldk, hk;
    void* k_out;               /* likewise; may be k with its pitches; NULL where a cache takes the rows */
    int64_t ldko, hko;
    const void* q_norm;        /* bf16 [head_dim]: the norms' weights; NULL: no norm */
    const void* k_norm;
    float eps;                 /* >= 0 */
    const int32_t* pos;        /* [tokens]: position of each token; NULL: no rotation, and the rest is ignored */
    const float* cos_t;        /* as in nvfp4_rope_t */
    const float* sin_t;
    int64_t table_ld, positions;
    int64_t rope_dim;          /* the LAST rope_dim columns of a head are rotated; even, <= head_dim */
    int32_t halves;            /* pairs: 0 (2i, 2i+1); else (i, i + rope_dim/2), rope_dim % 16 == 0, of those columns */
    /* a cache that takes the k rows and those of v (slot NULL: none) */
    const int32_t* slot;       /* [tokens], as in nvfp4_kv_append */
    const void* v;             /* bf16 [tokens][kv_heads][head_dim] */
    int64_t ldv, hv;
    const nvfp4_kv_cache_t* cache;     /* one of the two */
    const nvfp4_kv4_cache_t* cache4;
} nvfp4_heads_t;

/*
 * nvfp4_qk_norm_rope -- RMSNorm of each query and key head and their rotary
 * embedding in one pass, for a token's heads x of q or k:
 *   y = x * (1 / sqrt(mean(x^2) + eps)) * norm           (or x without a norm)
 *   each pair (a, b) of the rotated columns:  a' = a*c - b*s,  b' = a*s + b*c
 * in binary32, rounded to bf16 once at the end.  Without a norm each product, sum
 * and difference is one operation (nvfp4_gemm_rope's bits).  With one the weights
 * are folded into c and s, the sums fused and 1 / rms applied last: before the last
 * rounding within 2^-18 of the sum of the products' magnitudes.  A row whose squares
 * are beyond binary32 becomes 0, an infinity in it (and, rotated, its partner) NaN.
 * c and s are those of the pair in row pos[t] of the tables; a position outside
 * them takes the nearest row and records NVFP4_ERR_INVALID_ARG * 100 + 33.
 * With a cache the rows of k, rounded to bf16, and those of v go where
 * nvfp4_kv_append (or nvfp4_kv4_append) would put them, bit for bit; k_out may
 * then be NULL.
 */
int nvfp4_qk_norm_rope(const nvfp4_heads_t* heads, nvfp4_stream_t stream);

/* ------------------------------------------------- a KV cache in 4 bits
 *
 * Rows of the paged cache as NVFP4: 9/32 of the bf16 cache's bytes, which is
 * what a decode step reads.
 */

/* Page p, kv head h, row i of K: codes (two columns to a byte, the even one in
 * the low nibble) at k + p*page_stride + (h*page_size + i)*head_dim/2, one E4M3
 * scale per 16 columns at k_sf + p*sf_stride + (h*page_size + i)*head_dim/16;
 * column value = E2M1(code) * E4M3(scale) * *k_g.  V likewise. */
struct nvfp4_kv4_cache {
    uint8_t* k;                /* 16-byte aligned */
    uint8_t* v;
    uint8_t* k_sf;
    uint8_t* v_sf;
    const float* k_g;          /* [1], device: 2^-80 .. 2^120; e.g. a power of two near max |k| / 2688 */
    const float* v_g;
    int64_t pages, page_size, kv_heads;
    int64_t head_dim;          /* 16 .. 128, % 16 == 0 */
    int64_t page_stride;       /* bytes, >= kv_heads*page_size*head_dim/2, % 16 == 0, below 2^32 */
    int64_t sf_stride;         /* bytes, >= kv_heads*page_size*head_dim/16, % 16 == 0, below 2^32 */
};

/*
 * nvfp4_kv4_append -- nvfp4_kv_append into a 4-bit cache: each 16 columns
 * quantized as nvfp4_quantize does with the global scale *k_g (*v_g):
 *   s = E4M3(amax16 / (6*g)),  code = s == 0 ? +0 : E2M1(x / (E4M3(s) * g)).
 * Infinities count as the largest bf16 number (beyond 448*6*g a block's scale
 * is 448, and a value beyond 6 times that scale is 6 times it); a block with a
 * NaN gets the scale NaN and the codes 0.  Slots as in nvfp4_kv_append.
 */
int nvfp4_kv4_append(const void* k, int64_t ldk, int64_t hk, const void* v, int64_t ldv, int64_t hv,
                     const int32_t* slot, int64_t tokens, const nvfp4_kv4_cache_t* cache, nvfp4_stream_t stream);

/*
 * nvfp4_kv4_expand -- the rows of a 4-bit cache that a step's new tokens see
 * (request r: positions max(0, kv_len - q_len - window + 1) .. kv_len - 1; none
 * where q_len is 0), as bf16 into the same pages and rows of `out`; its other rows stay as they are.  The
 * value is rounded to bf16 once (exact where *k_g is a power of two).
 *   step     after nvfp4_attn_plan on the same stream order; its window counts
 *            if it has heads.
 *   out      pages, page_size, kv_heads and head_dim of `cache`.
 * Entries of the block table outside the cache are skipped.
 */
int nvfp4_kv4_expand(const nvfp4_kv4_cache_t* cache, const nvfp4_step_t* step, const nvfp4_kv_cache_t* out,
                     nvfp4_stream_t stream);

/*
 * nvfp4_attn_paged4 -- nvfp4_attn_paged over a 4-bit cache, whose values it
 * takes as they are stored (in half precision, which holds code times scale
 * exactly; *k_g and *v_g multiply the scores and the outputs).  q counts with
 * at least 11 bits beside the largest of its row, the probabilities are rounded
 * to half precision (2^-11; one below 2^-20 of its row's largest by 2^-31 of that).
 *   expanded  NULL, or a bf16 cache of the same pages, page_size, kv_heads and
 *            head_dim as scratch: a step with many rows per request then takes
 *            its keys' rows out of the 4 bits once (into their pages there, 16 bits
 *            that hold code times scale exactly) and runs nvfp4_attn_paged's
 *            kernel on them, q as it is and probabilities in half precision too (scores
 *            below 2^24 keep their largest there, straight from the codes those of any
 *            size).  That is so with 40 rows (tokens, padding included, times heads /
 *            kv_heads) per request or more on average, else never with as many tokens as
 *            requests, and in between where the lengths want more than a few passes over
 *            the keys, of all requests or of one (the plan's schedule has that; two of
 *            the three launches then return at once or one does).
 *            One serves all layers that run one after the other.
 *   workspace as nvfp4_attn_paged.
 * head_dim % 16 == 0.  The rest as nvfp4_attn_paged: cache rows that no row of
 * a request sees may hold anything, a page id outside the cache counts as a
 * page of zeros.
 */
int nvfp4_attn_paged4(const nvfp4_step_t* step, const nvfp4_attn_io_t* io, const nvfp4_kv4_cache_t* cache,
                      const nvfp4_kv_cache_t* expanded, void* workspace, size_t workspace_bytes,
                      nvfp4_stream_t stream);

/* ------------------------------------------------------ pages of a cache
 *
 * Requests that fork, pages that come free, pages moved together.  A page is in
 * use while a request holds it: request r holds the first
 * ceil(ctx_len[r] / page_size) entries of its row of the block table.  Requests
 * may share pages; one has ended when its ctx_len is 0.  No counts are kept.
 */

typedef struct {
    int32_t* block_table;      /* [R x table_cols], row pitch table_ld */
    int64_t requests;          /* R, 1 .. 8192 */
    int64_t table_cols, table_ld;
    int32_t* ctx_len;          /* [R] tokens in the cache */
    int64_t page_size;         /* 16, 32, 64 or 128 */
    int64_t pages;             /* of the caches, 1 .. 2^20 */
} nvfp4_pages_t;

/*
 * nvfp4_pages_fork -- request dst[i] becomes a copy of request src[i], i < n:
 * it gets its length and shares its full pages.  A last page that is not full,
 * which both will write, becomes one of free_pages[*cursor ..] (pair after
 * pair), and (its source, itself) are (copy_src[i], copy_dst[i]) for
 * nvfp4_pages_copy, -1 where nothing is to be copied.  The rest of dst's row
 * becomes -1.
 *   src, dst   int32 [n], device; n <= requests.  A pair with a request that
 *              does not exist, a dst that is some pair's src or an earlier
 *              pair's dst, or a src whose length its row cannot hold, is
 *              left out.
 *   cursor     [1] entries of free_pages already taken, or NULL: 0; cursor_out
 *              [1] or NULL: that plus the pages taken, may alias cursor.
 *   copy_src, copy_dst   int32 [n], device, out.
 * A pair left out, and a page that the free list did not have or that is no page
 * (the entry is -1), record NVFP4_ERR_INVALID_ARG * 100 + 34.
 */
int nvfp4_pages_fork(const nvfp4_pages_t* pages, const int32_t* src, const int32_t* dst, int64_t n,
                     const int32_t* free_pages, int64_t free_count, const int32_t* cursor, int32_t* cursor_out,
                     int32_t* copy_src, int32_t* copy_dst, nvfp4_stream_t stream);

/*
 * nvfp4_pages_free -- the free list from what the requests hold: the pages that
 * none of them holds, ascending, then -1, into free_pages (int32 [pages]; the
 * next step's list, its cursor at 0), their number into *free_count.  With
 * table_out the pages in use are moved together as well: those at or past their
 * number take the lowest free ids, in order.  (move_src[i], move_dst[i]), int32
 * [pages / 2] each, -1 past the last, are the moves for nvfp4_pages_copy;
 * table_out (row pitch table_out_ld; may be the table itself) gets the rows with
 * the new ids, -1 past what a request holds; and the free list is that after the
 * moves.  Lengths and block_table are not changed.
 * A held entry that is no page is left as it is and recorded
 * (NVFP4_ERR_INVALID_ARG * 100 + 34), as is a length that its row cannot hold.
 */
int nvfp4_pages_free(const nvfp4_pages_t* pages, int32_t* free_pages, int32_t* free_count, int32_t* table_out,
                     int64_t table_out_ld, int32_t* move_src, int32_t* move_dst, nvfp4_stream_t stream);

/* One matrix of pages: page p is page_bytes bytes at base + p*page_stride
 * (16-byte aligned, both % 16 == 0): K or V of a cache, codes or scales. */
typedef struct {
    void* base;
    int64_t page_bytes, page_stride;
} nvfp4_plane_t;

/*
 * nvfp4_pages_copy -- page src[i] to page dst[i], i < n, in every plane (the
 * caches of all layers in one call).  A pair of -1 is skipped; any other id
 * outside [0, pages) skips its pair and records NVFP4_ERR_INVALID_ARG * 100 + 34.
 * No page is the destination of two pairs, or source and destination
 * of different ones.
 *   planes   HOST array; up to 64 to a launch.
 *   src, dst int32 [n], device.
 */
int nvfp4_pages_copy(const nvfp4_plane_t* planes, int64_t n_planes, int64_t pages, const int32_t* src,
                     const int32_t* dst, int64_t n, nvfp4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_H */

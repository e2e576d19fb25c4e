/*
 * gbln.h -- C ABI of the GB300 (sm_103a) layer-operator library libgbln.so.
 *
 * Operators: RMSNorm with fused residual add (forward, backward, weight-gradient
 * finalize), rotary position embedding on Q and K (forward, backward, cos/sin
 * table, per-document positions) and SwiGLU (forward, backward); LayerNorm,
 * other gated and plain activations, MXFP8 and row-scaled FP8 outputs for the
 * next GEMM, 8-bit activation checkpoints with the backward passes that read
 * them, and a quantised K/V cache; per-head norms of Q and K with the rotation in
 * one pass, rotary embedding with several position axes, and attention over the
 * quantised cache.
 *
 * Sources that name these operators (they print no formulas; the standard
 * definitions are used and written out at each entry point):
 *   [FL]  "Fast-LLM: 高效大语言模型训练框架", §三 技术架构: table "Transformer Block
 *         结构" (Normalization LayerNorm / RMSNorm; attention + RoPE; MLP gated or
 *         not, SiLU / GeLU / ReLU) and "训练配置示例" (rms_norm with epsilon;
 *         rotary type default with theta; gated MLP with activation silu;
 *         micro_batch_size in tokens with maximum_document_length).
 *   [LF]  "LLaMA-Factory Kernels 系统": the fused RMSNorm, SwiGLU and RoPE operators.
 *   [HF]  "Kernels（自定义内核）", §Liger: RMSNorm, RoPE and SwiGLU fused into single
 *         kernels for training; fusion saves memory traffic and launches.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Memory: every pointer is DEVICE memory on the current CUDA device, owned and
 *    allocated by the caller.  The library never allocates and never frees.  Its
 *    only state is per device: the SM count, the device error word, flags that
 *    record which kernels' shared-memory limits have been raised, and the fixed
 *    scratch array of gbln_rmsnorm_bwd_noalloc.  It tracks 64 devices: on a
 *    device with ordinal 64 or above, the calls that need that state (the
 *    backward passes, RoPE, the gated units and activations, the error word)
 *    return GBLN_ERR_CUDA.  That state is looked up once per device and kept for
 *    the life of the process, so the device's primary context must not be torn
 *    down (cudaDeviceReset, or the driver API's primary-context reset) while the
 *    library is in use: after a reset the cached addresses (error word, scratch
 *    array) and shared-memory limits no longer hold.
 *  - Layout: row-major and contiguous.  "[T, H]" means T rows of H elements.
 *  - Streams: work is enqueued on `stream` (NULL = the legacy default stream) and
 *    the call returns without synchronising.  Errors raised by the kernels
 *    themselves appear on the stream, not in the returned status.
 *  - CUDA graphs: every call can be captured.  The first call of an entry point
 *    on a device does one-time set-up (SM count, the device error word's
 *    address, kernel shared-memory limits); make that first call outside
 *    stream capture.
 *  - Types: `io` is the element type of activations and gradients, `wt` the type
 *    of the RMSNorm weight.  Supported: io = wt = F32; io = wt = BF16;
 *    io = BF16 with wt = F32.  Arithmetic is float32; bf16 results are rounded
 *    to nearest even once.
 *  - Alignment: any alignment is accepted.  Pointers aligned to 16 bytes with
 *    row widths that are a multiple of 16 bytes take the 128-bit vector path;
 *    anything else takes a slower element-wise path of the same kernels.
 *  - Errors: arguments are checked on the host before any CUDA call.  A null
 *    required pointer, a negative or out-of-range size, eps < 0 or not finite,
 *    an odd head size, theta <= 0, or a workspace that is too small returns an
 *    error and launches nothing.  T == 0 returns GBLN_OK and launches nothing
 *    once sizes, scalars and dtypes pass; its pointers are not examined (empty
 *    tensors may have null data pointers).  A failed launch returns GBLN_ERR_CUDA.
 *  - Aliasing: outputs may alias their own input exactly where an entry point
 *    says so; partial overlap is undefined.
 */
#ifndef GBLN_H
#define GBLN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream; declared here so that no CUDA header is needed. */
typedef struct CUstream_st* gbln_stream_t;

typedef enum {
  GBLN_OK = 0,
  GBLN_ERR_INVALID_ARG = 1, /* null pointer, bad size, bad scalar                */
  GBLN_ERR_UNSUPPORTED = 2, /* dtype combination outside the supported set       */
  GBLN_ERR_WORKSPACE = 3,   /* dW partial workspace smaller than required        */
  GBLN_ERR_CUDA = 4         /* a CUDA runtime call or launch failed              */
} gbln_status;

typedef enum { GBLN_F32 = 0, GBLN_BF16 = 1 } gbln_dtype;

/* Activation of the gated and plain MLP units ([FL] 支持的 MLP 变体: SiLU / GeLU / ReLU). */
typedef enum {
  GBLN_ACT_SILU = 0,      /* x / (1 + exp(-x))                                    */
  GBLN_ACT_GELU_TANH = 1, /* 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3)))       */
  GBLN_ACT_GELU_ERF = 2,  /* 0.5 x (1 + erf(x / sqrt(2)))  (exact GeLU)             */
  GBLN_ACT_RELU = 3       /* max(x, 0); derivative 1 for x > 0, else 0              */
} gbln_act;

/* Human-readable name of a status code.  Never NULL; the string is static. */
const char* gbln_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int gbln_version(void);

/*
 * Per-device error word of the current device, a set of bits:
 *   1  a kernel's bounded wait on its own asynchronous (TMA bulk) copies, or
 *      (attention) on another part of its block, ran out; instead of hanging the
 *      kernel stopped early, or (attention) ran on to its end with what it had,
 *      all of it in bounds: its outputs are not valid;
 *   2  a RoPE call met a position outside [0, max_pos); that token's outputs
 *      are NaN (the table is not read);
 *   4  a cache call met a slot beyond the cache's last one (nothing was stored
 *      for that token, its read-back is NaN), or attention a page outside the
 *      cache (the rows that see it are NaN).
 * *code receives the word; clear != 0 resets it to zero.  Synchronous
 * (device-wide copy): call it outside hot loops.  Errors: INVALID_ARG for a
 * null code, CUDA if the device is unreachable.
 */
gbln_status gbln_device_error(uint32_t* code, int clear);

/*
 * Self-test of the timeout path: launches one thread that waits, with the
 * bounded poll loop of the TMA pipelines, on a barrier nothing completes; after
 * `polls` polls (1 <= polls <= 2^22) it sets bit 1 of the device error word and
 * returns.  Touches no caller memory; the context stays usable.  For tests.
 */
gbln_status gbln_selftest_wait_timeout(uint32_t polls, gbln_stream_t stream);

/* ------------------------------------------------------------------------- */
/* RMSNorm with fused residual add ([FL] Transformer Block 结构, 训练配置示例;  */
/* [LF] fused RMSNorm; [HF] §Liger)                                          */
/* ------------------------------------------------------------------------- */

/*
 * Forward, per row t of T rows of H channels:
 *   h[t]    = x[t] + residual[t]           (rounded to io; h = x when residual is NULL)
 *   rstd[t] = 1 / sqrt(mean_j h[t,j]^2 + eps)
 *   y[t,j]  = weight[j] * h[t,j] * rstd[t]  (one rounding to io)
 *
 * x, residual      [T, H] io, read.  residual may be NULL (plain RMSNorm).
 * weight           [H] wt, read.
 * y                [T, H] io, written.
 * residual_out     [T, H] io, written with h.  Required iff residual != NULL,
 *                  ignored otherwise.  May alias x or residual exactly.
 * rstd             [T] float32, written; the backward pass reads it.
 * eps              >= 0 and finite.
 * Errors: INVALID_ARG for null x/weight/y/rstd, T < 0, H <= 0, H > 2^24, bad eps,
 *         missing residual_out; UNSUPPORTED for other dtype pairs.
 */
gbln_status gbln_rmsnorm_fwd(const void* x, const void* residual, const void* weight,
                             void* y, void* residual_out, float* rstd,
                             int64_t T, int64_t H, float eps,
                             gbln_dtype io, gbln_dtype wt, gbln_stream_t stream);

/*
 * Rows of the float32 weight-gradient workspace that gbln_rmsnorm_bwd writes
 * for this shape on the current device: the workspace is [P, H] float32.
 * P depends only on (T, H, io) and the device's SM count, so a fixed shape on a
 * fixed GPU model always uses the same P and the same summation order.
 * Returns P >= 1 for T >= 1, 0 for T == 0, and -1 on invalid arguments or when
 * the device cannot be queried.
 */
int64_t gbln_rmsnorm_bwd_num_partials(int64_t T, int64_t H, gbln_dtype io);

/*
 * Backward, first of two passes.  With n = h * rstd and g = dy * weight, per row:
 *   dx[t]  = rstd[t] * (g - n * mean_j(g[j] * n[j])) + dresidual_out[t]
 *   partial[p, j] = sum over the rows of block p of dy[t,j] * n[t,j]
 * dx is the gradient of both x and residual of the forward call.
 *
 * dy               [T, H] io, gradient of y.
 * dresidual_out    [T, H] io, gradient arriving on residual_out; NULL = zero.
 * h                [T, H] io, the forward's residual_out (or x if it had no residual).
 * weight           [H] wt.   rstd [T] float32 from the forward.
 * dx               [T, H] io, written.  May alias dy or dresidual_out exactly.
 * dw_partial       [P_cap, H] float32 workspace, rows 0..P-1 written, where
 *                  P = gbln_rmsnorm_bwd_num_partials(T, H, io).
 * P_cap            rows available in dw_partial; GBLN_ERR_WORKSPACE if P_cap < P.
 * The rows of a block and their order are fixed by (T, H, io, SM count): the
 * result is bitwise reproducible run to run.
 */
gbln_status gbln_rmsnorm_bwd(const void* dy, const void* dresidual_out, const void* h,
                             const void* weight, const float* rstd,
                             void* dx, float* dw_partial, int64_t P_cap,
                             int64_t T, int64_t H,
                             gbln_dtype io, gbln_dtype wt, gbln_stream_t stream);

/*
 * Backward, second pass: dw[j] = (accumulate ? dw[j] : 0) + sum_{p<P} partial[p, j],
 * summed in a fixed order (bitwise reproducible).
 * dw_partial [P, H] float32 as written by gbln_rmsnorm_bwd, P exactly the value
 * gbln_rmsnorm_bwd_num_partials returned for that call.  dw [H] float32.
 */
gbln_status gbln_rmsnorm_dw_finalize(const float* dw_partial, int64_t P, int64_t H,
                                     float* dw, int accumulate, gbln_stream_t stream);

/*
 * Backward without a caller-provided workspace: dx as gbln_rmsnorm_bwd, and the
 * finished weight gradient dw [H] float32 (as gbln_rmsnorm_dw_finalize with
 * accumulate = 0), in two launches on `stream`.  The sources have no
 * counterpart of this entry point; it exists for callers that cannot allocate
 * device memory where they run the backward pass (a region being recorded into
 * a CUDA graph under a capture mode that forbids cudaMalloc, a runtime whose
 * device memory belongs to a pool it may not bypass, a latency-critical loop in
 * which an allocation could synchronise the device).  The caller still passes
 * every input and output.
 *
 * Scratch: the dW partial rows live in one fixed array inside the library
 * (4 Mi float32 = 16 MiB, held by every GPU that loads the library until the
 * process exits).  Every call on a device uses the same array and overwrites the
 * rows it reads, so nothing needs clearing; calls that may overlap on the GPU
 * (other streams, other threads) race on it and must be serialised by the caller.
 * The usual number of partial rows is reduced when it would not fit, so the
 * summation order (still fixed for a shape and GPU) can differ from
 * gbln_rmsnorm_bwd's by float32 rounding.
 * Set-up: the first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call before
 * any stream capture.  The address is kept until the process exits: resetting
 * the device's primary context (cudaDeviceReset) while the library is loaded
 * moves the array, and later calls would write through the stale address, so
 * do not reset a device that this entry point has been called on.
 * Errors: as gbln_rmsnorm_bwd; GBLN_ERR_WORKSPACE if H > 4 Mi (a partial row
 * would not fit); GBLN_ERR_CUDA if the address lookup fails.  T == 0 sets dw to
 * zero (one launch).  dx may alias dy or dresidual_out exactly.
 */
gbln_status gbln_rmsnorm_bwd_noalloc(const void* dy, const void* dresidual_out, const void* h,
                                     const void* weight, const float* rstd,
                                     void* dx, float* dw, int64_t T, int64_t H,
                                     gbln_dtype io, gbln_dtype wt, gbln_stream_t stream);

/* ------------------------------------------------------------------------- */
/* LayerNorm with fused residual add ([FL] Transformer Block 结构:             */
/* normalization LayerNorm / RMSNorm)                                         */
/* ------------------------------------------------------------------------- */

/*
 * Forward, per row t of H channels:
 *   h = x + residual (rounded to io; h = x when residual is NULL)
 *   mean[t] = mean_j h;  var = mean_j (h - mean)^2;  rstd[t] = 1 / sqrt(var + eps)
 *   y = weight * (h - mean) * rstd + bias  (bias NULL = no bias; one rounding to io)
 * Arguments as gbln_rmsnorm_fwd, plus bias [H] wt (nullable) and mean [T] float32
 * (written; the backward pass reads it with rstd).
 */
gbln_status gbln_layernorm_fwd(const void* x, const void* residual, const void* weight,
                               const void* bias, void* y, void* residual_out, float* mean,
                               float* rstd, int64_t T, int64_t H, float eps, gbln_dtype io,
                               gbln_dtype wt, gbln_stream_t stream);

/* Rows P of the [P, 2H] float32 dW|dB workspace of gbln_layernorm_bwd (as gbln_rmsnorm_bwd_num_partials). */
int64_t gbln_layernorm_bwd_num_partials(int64_t T, int64_t H, gbln_dtype io);

/*
 * Backward, first pass.  With n = (h - mean) * rstd and g = dy * weight, per row:
 *   dx = rstd * (g - mean_j g - n * mean_j(g * n)) + dresidual_out
 *   partial[p, 0:H]  = sum over the rows of block p of dy * n   (dW)
 *   partial[p, H:2H] = sum over the rows of block p of dy       (dB)
 * Arguments as gbln_rmsnorm_bwd, plus mean [T] from the forward; the workspace is
 * [P_cap, 2H] float32.  Bitwise reproducible for a fixed shape and GPU model.
 */
gbln_status gbln_layernorm_bwd(const void* dy, const void* dresidual_out, const void* h,
                               const void* weight, const float* mean, const float* rstd,
                               void* dx, float* dwdb_partial, int64_t P_cap, int64_t T, int64_t H,
                               gbln_dtype io, gbln_dtype wt, gbln_stream_t stream);

/* Second pass: dw[j] (+)= sum_p partial[p, j], db[j] (+)= sum_p partial[p, H + j], fixed order. */
gbln_status gbln_layernorm_dwdb_finalize(const float* dwdb_partial, int64_t P, int64_t H,
                                         float* dw, float* db, int accumulate,
                                         gbln_stream_t stream);

/* ------------------------------------------------------------------------- */
/* Rotary position embedding on Q and K ([FL] attention with RoPE, rotary     */
/* type default with theta; [LF] fused RoPE; [HF] §Liger)                     */
/* ------------------------------------------------------------------------- */

/*
 * Cos/sin table: cos_sin[p, i] = (cos(p * f_i), sin(p * f_i)) as two float32,
 * f_i = theta^(-2 i / D), for p in [0, max_pos) and i in [0, D/2).  Angles and
 * their cosines are evaluated in double precision on the device and rounded once
 * to float32.  cos_sin: [max_pos, D/2, 2] float32, written.
 * Errors: INVALID_ARG for null, max_pos < 0, D <= 0 or odd, theta <= 0 or not finite.
 */
gbln_status gbln_rope_table(float* cos_sin, int64_t max_pos, int32_t D, double theta,
                            gbln_stream_t stream);

/*
 * Forward rotation, rotate-half pairing.  For every token t, every head of q and
 * of k, and i < D/2, with (c, s) = cos_sin[positions[t], i]:
 *   out[i]       = x[i] * c - x[i + D/2] * s
 *   out[i + D/2] = x[i + D/2] * c + x[i] * s
 * q [T, Hq, D], k [T, Hk, D] io, read; q_out, k_out same shapes, written (may
 * alias q and k exactly: in place).  Hk may be 0 (k, k_out ignored).
 * positions [T] int32: the position of each token inside its document.  A position
 * outside [0, max_pos) is not read from the table: that token's outputs are NaN.
 * cos_sin as written by gbln_rope_table for the same D and some max_pos.
 */
gbln_status gbln_rope_fwd(const void* q, const void* k, void* q_out, void* k_out,
                          const int32_t* positions, const float* cos_sin, int64_t max_pos,
                          int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                          gbln_dtype io, gbln_stream_t stream);

/*
 * Backward: the transpose (= inverse) rotation applied to the incoming gradients:
 *   din[i]       = dout[i] * c + dout[i + D/2] * s
 *   din[i + D/2] = dout[i + D/2] * c - dout[i] * s
 * Same arguments as gbln_rope_fwd with (dq, dk) in and (dq_in, dk_in) out.
 */
gbln_status gbln_rope_bwd(const void* dq, const void* dk, void* dq_in, void* dk_in,
                          const int32_t* positions, const float* cos_sin, int64_t max_pos,
                          int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                          gbln_dtype io, gbln_stream_t stream);

/* Pairing of the rotated elements. */
typedef enum {
  GBLN_ROPE_HALF = 0,       /* (i, i + D/2): the default rotary type (gbln_rope_fwd)   */
  GBLN_ROPE_INTERLEAVED = 1 /* (2i, 2i + 1), frequency index i                        */
} gbln_rope_pairing;

/*
 * gbln_rope_fwd with strided rows and a choice of pairing: head row h of token t
 * of q starts at q + t * ld_q + h * D (elements), likewise for k, q_out, k_out
 * (ld_q, ld_q_out >= Hq * D; ld_k, ld_k_out >= Hk * D).  Q and K can thus be read
 * from, and written back into, one packed [T, (Hq + 2 Hk) * D] QKV projection
 * output (q = qkv, k = qkv + Hq * D, every ld = (Hq + 2 Hk) * D; in place with
 * q_out = q, k_out = k).  Interleaved pairing rotates elements (2i, 2i + 1) by
 * pos * theta^(-2i/D) with the same cos/sin table.  Errors as gbln_rope_fwd, plus
 * INVALID_ARG for a stride below its row width or an unknown pairing.
 */
gbln_status gbln_rope_fwd_ex(const void* q, const void* k, void* q_out, void* k_out,
                             const int32_t* positions, const float* cos_sin, int64_t max_pos,
                             int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_q,
                             int64_t ld_k, int64_t ld_q_out, int64_t ld_k_out,
                             gbln_rope_pairing pairing, gbln_dtype io, gbln_stream_t stream);

/* Backward of gbln_rope_fwd_ex (inverse rotation), same layout arguments. */
gbln_status gbln_rope_bwd_ex(const void* dq, const void* dk, void* dq_in, void* dk_in,
                             const int32_t* positions, const float* cos_sin, int64_t max_pos,
                             int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_dq,
                             int64_t ld_dk, int64_t ld_dq_in, int64_t ld_dk_in,
                             gbln_rope_pairing pairing, gbln_dtype io, gbln_stream_t stream);

/*
 * Positions of packed documents: positions[t] = t - cu_seqlens[d] for the document
 * d with cu_seqlens[d] <= t < cu_seqlens[d+1] ([FL] 训练配置示例: micro-batches
 * counted in tokens hold several documents of at most maximum_document_length).
 * cu_seqlens [ndoc + 1] int32, non-decreasing, cu_seqlens[0] = 0 and
 * cu_seqlens[ndoc] = T (caller's contract: violating it gives wrong but in-bounds
 * results).  positions [T] int32, written.
 */
gbln_status gbln_positions_from_cu_seqlens(const int32_t* cu_seqlens, int32_t ndoc,
                                           int32_t* positions, int64_t T,
                                           gbln_stream_t stream);

/* ------------------------------------------------------------------------- */
/* SwiGLU ([FL] 支持的 MLP 变体, 训练配置示例 gated + silu; [LF] fused SwiGLU;   */
/* [HF] §Liger)                                                              */
/* ------------------------------------------------------------------------- */

/*
 * out = silu(gate) * up = gate / (1 + exp(-gate)) * up, elementwise.
 * gate, up, out: [T, I] io.  out may alias gate or up exactly.
 */
gbln_status gbln_swiglu_fwd(const void* gate, const void* up, void* out,
                            int64_t T, int64_t I, gbln_dtype io, gbln_stream_t stream);

/*
 * With s = sigmoid(gate):
 *   dgate = dout * up * s * (1 + gate * (1 - s))
 *   dup   = dout * gate * s
 * dout, gate, up: [T, I] io, read.  dgate, dup: [T, I] io, written; dgate may
 * alias gate and dup may alias up exactly (in place).
 */
gbln_status gbln_swiglu_bwd(const void* dout, const void* gate, const void* up,
                            void* dgate, void* dup,
                            int64_t T, int64_t I, gbln_dtype io, gbln_stream_t stream);

/* ------------------------------------------------------------------------- */
/* Gated units with any activation and row strides; plain activations          */
/* ([FL] 支持的 MLP 变体: dense MLP gated or not, SiLU / GeLU / ReLU)           */
/* ------------------------------------------------------------------------- */

/*
 * out[t, j] = f(gate[t, j]) * up[t, j] for t < T, j < I, f = act (see gbln_act).
 * Row t of each tensor starts ld elements after row t - 1 (ld >= I), so gate and
 * up may be the two halves of one packed [T, 2I] projection output
 * (gate = p, up = p + I, ld_gate = ld_up = 2I).  With every ld = I and
 * act = GBLN_ACT_SILU this is gbln_swiglu_fwd.  out may alias gate or up exactly.
 * Errors: INVALID_ARG for a bad act, T < 0, I <= 0, ld < I, null pointers (T > 0).
 */
gbln_status gbln_glu_fwd(const void* gate, const void* up, void* out, int64_t T, int64_t I,
                         int64_t ld_gate, int64_t ld_up, int64_t ld_out, gbln_act act,
                         gbln_dtype io, gbln_stream_t stream);

/*
 * dgate = dout * up * f'(gate), dup = dout * f(gate), each with its own row
 * stride (a packed [T, 2I] gradient: dgate = q, dup = q + I, ld = 2I).  dgate may
 * alias gate and dup may alias up exactly.  Errors as gbln_glu_fwd.
 */
gbln_status gbln_glu_bwd(const void* dout, const void* gate, const void* up, void* dgate,
                         void* dup, int64_t T, int64_t I, int64_t ld_dout, int64_t ld_gate,
                         int64_t ld_up, int64_t ld_dgate, int64_t ld_dup, gbln_act act,
                         gbln_dtype io, gbln_stream_t stream);

/* y = f(x) over n contiguous elements (non-gated MLP); y may alias x. */
gbln_status gbln_act_fwd(const void* x, void* y, int64_t n, gbln_act act, gbln_dtype io,
                         gbln_stream_t stream);

/* dx = dy * f'(x) over n contiguous elements; dx may alias dy or x. */
gbln_status gbln_act_bwd(const void* dy, const void* x, void* dx, int64_t n, gbln_act act,
                         gbln_dtype io, gbln_stream_t stream);

/* ------------------------------------------------------------------------- */
/* MXFP8 outputs for the next projection GEMM ([HF] Kernels intro: fusing a    */
/* producer with its consumer's input conversion saves an HBM pass)            */
/* ------------------------------------------------------------------------- */

/*
 * MXFP8 as defined by the OCP Microscaling Formats (MX) v1.0 specification:
 * blocks of 32 consecutive values of a row share one scale 2^e, stored as an
 * E8M0 byte (e + 127); each value is stored as an E4M3 byte (1 sign, 4
 * exponent bits with bias 7, 3 mantissa bits; largest finite 448).  Here
 *   e     = floor(log2(max |v| over the block)) - 8, clamped to [-127, 127]
 *           (-127 for an all-zero block),
 *   code  = E4M3(v / 2^e), rounded to nearest even, saturating to +-448.
 * Blocks run along the last axis, the reduction axis of the GEMM that
 * consumes the tensor (y @ W^T), which is the operand layout of block-scaled
 * FP8 tensor-core GEMMs.  Scales are stored row-major, [T, N / 32]; a GEMM
 * library that wants another arrangement of the scale bytes needs a permutation.
 * The quantised value is computed in float32 from the unrounded result.
 */

/*
 * gbln_rmsnorm_fwd with y also (or only) delivered as MXFP8:
 * y_e4m3 [T, H] bytes and y_scale [T, H / 32] bytes, both written.  y [T, H] io
 * may be NULL (then only the MXFP8 copy is written).  H must be a multiple of
 * 32.  Other arguments, aliasing and errors as gbln_rmsnorm_fwd; INVALID_ARG
 * also for H % 32 != 0 or a null y_e4m3 / y_scale.  Any alignment is accepted.
 */
gbln_status gbln_rmsnorm_fwd_mxfp8(const void* x, const void* residual, const void* weight,
                                   void* y, uint8_t* y_e4m3, uint8_t* y_scale,
                                   void* residual_out, float* rstd, int64_t T, int64_t H,
                                   float eps, gbln_dtype io, gbln_dtype wt,
                                   gbln_stream_t stream);

/*
 * Gated unit forward delivered as MXFP8 only: out = f(gate) * up (as
 * gbln_glu_fwd, with row strides ld_gate, ld_up >= I for packed [T, 2I] inputs)
 * written as out_e4m3 [T, I] bytes (contiguous) and out_scale [T, I / 32] bytes.
 * I must be a multiple of 32.  Errors as gbln_glu_fwd; INVALID_ARG also for
 * I % 32 != 0.  Any alignment is accepted.
 */
gbln_status gbln_glu_fwd_mxfp8(const void* gate, const void* up, uint8_t* out_e4m3,
                               uint8_t* out_scale, int64_t T, int64_t I, int64_t ld_gate,
                               int64_t ld_up, gbln_act act, gbln_dtype io,
                               gbln_stream_t stream);

/* ------------------------------------------------------------------------- */
/* 8-bit storage with float32 scales: the next GEMM's operand, activation      */
/* checkpoints and the K/V cache ([HF] Kernels intro and §Liger: fusing a       */
/* producer with its consumer's conversion, training memory)                   */
/* ------------------------------------------------------------------------- */

/*
 * A group of values v shares one float32 scale; each value is one byte, an INT8
 * integer or an E4M3 code.  In float32, every operation rounded to nearest even:
 *   a     = max(max |v|, 2^-100)
 *   code  = nearest(v * (qmax / a))    to an integer (INT8, qmax = 127) or to E4M3
 *                                      (qmax = 448), ties to even
 *   scale = a / qmax                   value = code * scale
 * The codes of given values are therefore the same on every run and in any
 * float32 implementation of these steps.  An all-zero group has the scale
 * 2^-100 / qmax and codes 0.  A group that holds an infinity or a NaN gets the
 * scale NaN (its codes are unspecified): all of it reads back as NaN.
 * A value is off by at most a / 254 with INT8, by the larger of 2^-4 of itself and
 * a / 448 * 2^-10 with E4M3 (values below that last bound become 0), each plus 2^-21 of
 * itself for the float32 roundings.  INT8 is the closer one for values of one size,
 * E4M3 where a group holds outliers.
 */
typedef enum { GBLN_Q8_INT8 = 0, GBLN_Q8_E4M3 = 1 } gbln_q8;

/*
 * gbln_rmsnorm_fwd with y also (or only) delivered as E4M3 with one scale per row
 * (group = row), the operand of a row-scaled FP8 GEMM.  With u = weight * h in
 * float32, y = u * rstd; rstd cancels out of the codes:
 *   a = max(max_j |u_j|, 2^-100);  y_e4m3 = E4M3(u * (448 / a));  y_scale = a * rstd / 448
 * y_e4m3 [T, H] bytes and y_scale [T] float32, both written; y [T, H] io may be
 * NULL.  Any H and any alignment.  Other arguments, aliasing and errors as
 * gbln_rmsnorm_fwd; INVALID_ARG also for a null y_e4m3 / y_scale.
 */
gbln_status gbln_rmsnorm_fwd_fp8(const void* x, const void* residual, const void* weight,
                                 void* y, uint8_t* y_e4m3, float* y_scale, void* residual_out,
                                 float* rstd, int64_t T, int64_t H, float eps, gbln_dtype io,
                                 gbln_dtype wt, gbln_stream_t stream);

/*
 * Gated unit forward delivered as E4M3 with one scale per row only: the float32
 * result f(gate) * up (as gbln_glu_fwd, row strides ld_gate, ld_up >= I) quantised
 * with group = row.  out_e4m3 [T, I] bytes (contiguous), out_scale [T] float32.
 * Any I and any alignment; T < 2^31.  Errors as gbln_glu_fwd.
 */
gbln_status gbln_glu_fwd_fp8(const void* gate, const void* up, uint8_t* out_e4m3,
                             float* out_scale, int64_t T, int64_t I, int64_t ld_gate,
                             int64_t ld_up, gbln_act act, gbln_dtype io, gbln_stream_t stream);

/*
 * Activation checkpoints: what a backward pass needs of its forward's input, kept
 * in 8 bits.  A group is 128 consecutive values of a row (the last one of a row may be
 * shorter): a [T, N] tensor becomes [T, N] bytes and [T, ceil(N / 128)] float32, both
 * contiguous, 1.03 bytes per value.
 */

/*
 * gbln_rmsnorm_fwd that also writes the checkpoint of h (= x + residual rounded to io,
 * or x) in the same pass: h8 [T, H] bytes, h8_scale [T, ceil(H / 128)] float32.  y, h
 * and rstd as gbln_rmsnorm_fwd: h to the bit; rstd may differ from it by the rounding of
 * the row's sum, which these kernels take in another order where rows are unaligned or
 * wide, and y with it.  Any H and alignment.  Arguments, aliasing and errors as
 * gbln_rmsnorm_fwd; INVALID_ARG also for an unknown fmt or a null h8 / h8_scale.
 */
gbln_status gbln_rmsnorm_fwd_ckpt8(const void* x, const void* residual, const void* weight,
                                   void* y, void* residual_out, float* rstd, uint8_t* h8,
                                   float* h8_scale, int64_t T, int64_t H, float eps, gbln_q8 fmt,
                                   gbln_dtype io, gbln_dtype wt, gbln_stream_t stream);

/* Rows P of the [P, H] float32 dW workspace of gbln_rmsnorm_bwd_ckpt8 (as gbln_rmsnorm_bwd_num_partials). */
int64_t gbln_rmsnorm_bwd_ckpt8_num_partials(int64_t T, int64_t H, gbln_dtype io);

/*
 * gbln_rmsnorm_bwd with h read from its checkpoint: n = (h8 * h8_scale) * rstd, the rest
 * as there (rstd is the forward's, of the exact h).  dw_partial is finished by
 * gbln_rmsnorm_dw_finalize.  dx may alias dy or dresidual_out exactly.  Bitwise
 * reproducible for a fixed shape, alignment and GPU model.  Errors as gbln_rmsnorm_bwd;
 * INVALID_ARG also for an unknown fmt or a null h8 / h8_scale.
 */
gbln_status gbln_rmsnorm_bwd_ckpt8(const void* dy, const void* dresidual_out, const uint8_t* h8,
                                   const float* h8_scale, const void* weight, const float* rstd,
                                   void* dx, float* dw_partial, int64_t P_cap, int64_t T,
                                   int64_t H, gbln_q8 fmt, gbln_dtype io, gbln_dtype wt,
                                   gbln_stream_t stream);

/*
 * gbln_glu_fwd that also writes the checkpoints of gate and up in the same pass:
 * gate8, up8 [T, I] bytes and gate_scale, up_scale [T, ceil(I / 128)] float32, all
 * contiguous.  out may alias gate or up exactly: their checkpoints are of the values
 * read.  Any I and alignment.  Errors as gbln_glu_fwd; INVALID_ARG also for an unknown
 * fmt or a null checkpoint pointer.
 */
gbln_status gbln_glu_fwd_ckpt8(const void* gate, const void* up, void* out, uint8_t* gate8,
                               float* gate_scale, uint8_t* up8, float* up_scale, int64_t T,
                               int64_t I, int64_t ld_gate, int64_t ld_up, int64_t ld_out,
                               gbln_act act, gbln_q8 fmt, gbln_dtype io, gbln_stream_t stream);

/*
 * gbln_glu_bwd with gate and up read from their checkpoints: with g = gate8 * gate_scale
 * and u = up8 * up_scale, dgate = dout * u * f'(g), dup = dout * f(g).  dout, dgate and dup
 * may be strided rows (each ld >= I).  dgate or dup may alias dout exactly.  Errors as
 * gbln_glu_bwd; INVALID_ARG also for an unknown fmt.
 */
gbln_status gbln_glu_bwd_ckpt8(const void* dout, const uint8_t* gate8, const float* gate_scale,
                               const uint8_t* up8, const float* up_scale, void* dgate, void* dup,
                               int64_t T, int64_t I, int64_t ld_dout, int64_t ld_dgate,
                               int64_t ld_dup, gbln_act act, gbln_q8 fmt, gbln_dtype io,
                               gbln_stream_t stream);

/*
 * One 8-bit cache (of K, or of V): `pages` pages of `page_size` slots, a slot holding
 * one token: Hk heads of D bytes and Hk scales.  Slot s is slot s % page_size of page
 * s / page_size.  Head h of slot o of page p starts at
 *   codes + p * page_stride + o * slot_stride + h * head_stride               (bytes)
 *   scale + p * scale_page_stride + o * scale_slot_stride + h * scale_head_stride (floats)
 * so pages may be [page_size, Hk, D] or [Hk, page_size, D], and K and V may be
 * interleaved in one allocation.  The strides must keep pages, slots and heads apart, and
 * K's from V's where they are written.
 */
typedef struct {
  uint8_t* codes;
  float* scale;
  int64_t pages, page_size;
  int64_t page_stride, slot_stride, head_stride;
  int64_t scale_page_stride, scale_slot_stride, scale_head_stride;
} gbln_cache8;

/*
 * gbln_rope_fwd_ex for serving: rotates q and k by their tokens' positions, and
 * instead of writing k back quantises the rotated k (float32, unrounded) and v into
 * their caches at the tokens' slots; a group is one head of one token.
 * A rotated pair is fmaf(x1, c, -(x2 s)), fmaf(x2, c, x1 s) in float32, whatever the sizes,
 * strides and alignment: the stored bits of a token do not depend on how a prompt is cut.
 * (gbln_rope_fwd_ex leaves these roundings to its kernels: its values may differ by one.)
 * q [T, Hq, D], k, v [T, Hk, D] io with token strides ld_q, ld_k, ld_v (e.g. inside one
 * packed QKV row); q_out as q with ld_q_out (may alias q exactly).  Hq may be 0 (q and
 * q_out ignored); Hk >= 1.
 * positions [T] int32, cos_sin as gbln_rope_fwd.  A position outside [0, max_pos): q_out
 * is NaN, k's scales are NaN, v is stored as usual, bit 2 of the error word is set.
 * slots [T] int64, distinct where they are not negative: token t goes to slot slots[t];
 * a negative one is padding (nothing is stored, its position matters only if Hq > 0); one
 * at or beyond pages * page_size stores nothing and sets bit 4.  Slots not named keep
 * their contents.  With two tokens on one slot, that slot's contents are unspecified.
 * k_cache, v_cache: host structs, read during the call; same pages and page_size.
 * Errors: INVALID_ARG as gbln_rope_fwd_ex, and for Hk < 1, an unknown fmt, a null or
 * inconsistent cache, strides that let pages, slots or heads overlap, K and V caches at
 * one address; CUDA.
 */
gbln_status gbln_rope_fwd_cache8(const void* q, const void* k, const void* v, void* q_out,
                                 const int32_t* positions, const float* cos_sin, int64_t max_pos,
                                 const int64_t* slots, const gbln_cache8* k_cache,
                                 const gbln_cache8* v_cache, int64_t T, int32_t Hq, int32_t Hk,
                                 int32_t D, int64_t ld_q, int64_t ld_k, int64_t ld_v,
                                 int64_t ld_q_out, gbln_rope_pairing pairing, gbln_q8 fmt,
                                 gbln_dtype io, gbln_stream_t stream);

/*
 * Read-back: k_out[t] and v_out[t] [Hk, D] io = the values of slot slots[t] (code * scale,
 * rounded once to io), for t < T in any order and with repeats.  A negative slot gives
 * zeros; one at or beyond pages * page_size gives NaN and sets bit 4 of the error word.
 * ld_k_out, ld_v_out >= Hk * D.  Errors as gbln_rope_fwd_cache8.
 */
gbln_status gbln_cache8_read(const int64_t* slots, const gbln_cache8* k_cache,
                             const gbln_cache8* v_cache, void* k_out, void* v_out, int64_t T,
                             int32_t Hk, int32_t D, int64_t ld_k_out, int64_t ld_v_out,
                             gbln_q8 fmt, gbln_dtype io, gbln_stream_t stream);

/* ------------------------------------------------------------------------- */
/* Between the QKV projection and attention: per-head RMSNorm of Q and K, rotary */
/* embedding with several position axes, attention over the 8-bit cache          */
/* ([FL] attention with RoPE, heads / head_groups; [LF] fused RMSNorm, fused     */
/* RoPE; [HF] §Liger: one pass instead of two)                                   */
/* ------------------------------------------------------------------------- */

/*
 * Position axes.  A token has n_axes positions (1 to 4; e.g. time, height, width), row a
 * of positions [n_axes, T] int32 starting at positions + a * ld_positions (ld_positions >=
 * T), and pair i of a head turns by its own axis' position:
 *   (c, s) = cos_sin[positions[axis[i]][t], i].
 * axis: HOST array of D / 2 bytes, each below n_axes, read during the call.  With n_axes
 * = 1 axis and ld_positions are ignored: the plain rotary embedding.  cos_sin is
 * gbln_rope_table's, or any table of its layout (axes with frequencies of their own).
 * A token with any of its positions outside [0, max_pos) gets NaN and sets bit 2 of the
 * error word.
 *
 * The five calls below take even D up to 512, any strides and alignment, and heads of q
 * and k at t * ld + h * D as gbln_rope_fwd_ex; Hk may be 0 (k ignored).  Aligned rows
 * (16 bytes, or 8 for bf16 heads such as 72) take the vector path.
 */

/* Rotation of q and k (gbln_rope_fwd_ex with position axes); in place allowed. */
gbln_status gbln_rope_axes_fwd(const void* q, const void* k, void* q_out, void* k_out,
                               const int32_t* positions, int64_t ld_positions, int32_t n_axes,
                               const uint8_t* axis, const float* cos_sin, int64_t max_pos,
                               int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_q,
                               int64_t ld_k, int64_t ld_q_out, int64_t ld_k_out,
                               gbln_rope_pairing pairing, gbln_dtype io, gbln_stream_t stream);

/* Its backward: the inverse rotation of the gradients; in place allowed. */
gbln_status gbln_rope_axes_bwd(const void* dq, const void* dk, void* dq_in, void* dk_in,
                               const int32_t* positions, int64_t ld_positions, int32_t n_axes,
                               const uint8_t* axis, const float* cos_sin, int64_t max_pos,
                               int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_dq,
                               int64_t ld_dk, int64_t ld_dq_in, int64_t ld_dk_in,
                               gbln_rope_pairing pairing, gbln_dtype io, gbln_stream_t stream);

/*
 * RMSNorm of every head of q and of k, then the rotation, in one pass.  For one head x:
 *   u = (x * rstd) * w,  rstd = 1 / sqrt(mean_D x^2 + eps),  out = rotation of u
 * rounded once to io.  q_weight, k_weight [D] wt are shared by the heads.  q_out may alias
 * q and k_out k exactly (a training step keeps them: the backward pass reads q and k).
 * Errors: UNSUPPORTED for other dtype pairs than gbln_rmsnorm_fwd's; INVALID_ARG as
 * gbln_rope_fwd_ex, for D > 512, bad axes, eps < 0 or not finite, null weights.
 */
gbln_status gbln_qk_norm_rope_fwd(const void* q, const void* k, const void* q_weight,
                                  const void* k_weight, void* q_out, void* k_out,
                                  const int32_t* positions, int64_t ld_positions, int32_t n_axes,
                                  const uint8_t* axis, const float* cos_sin, int64_t max_pos,
                                  int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_q,
                                  int64_t ld_k, int64_t ld_q_out, int64_t ld_k_out, float eps,
                                  gbln_rope_pairing pairing, gbln_dtype io, gbln_dtype wt,
                                  gbln_stream_t stream);

/*
 * Rows P of the [P, 2 D] float32 dWq|dWk workspace of gbln_qk_norm_rope_bwd: by the sizes
 * and the device's SM count alone.  0 for T == 0, -1 on invalid arguments.
 */
int64_t gbln_qk_norm_rope_bwd_num_partials(int64_t T, int32_t Hq, int32_t Hk, int32_t D);

/*
 * Backward of gbln_qk_norm_rope_fwd, first of two passes.  q and k are the forward's
 * inputs (rstd is recomputed from them), dq and dk the gradients of its outputs.  With d =
 * dq turned back, g = d * w, n = x * rstd, per head:
 *   dq_in = rstd * (g - n * mean_D(g * n))
 *   partial[p, 0:D] = sum over the heads of q of block p of d * n, [D:2D] the same of k
 * dq_in may alias dq or q exactly, dk_in dk or k.  dw_partial [P_cap, 2 D] float32, rows
 * 0..P-1 written; WORKSPACE if P_cap < P.  Bitwise reproducible for fixed sizes, alignment
 * and GPU model.  Errors as the forward.
 */
gbln_status gbln_qk_norm_rope_bwd(const void* dq, const void* dk, const void* q, const void* k,
                                  const void* q_weight, const void* k_weight, void* dq_in,
                                  void* dk_in, float* dw_partial, int64_t P_cap,
                                  const int32_t* positions, int64_t ld_positions, int32_t n_axes,
                                  const uint8_t* axis, const float* cos_sin, int64_t max_pos,
                                  int64_t T, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_dq,
                                  int64_t ld_dk, int64_t ld_q, int64_t ld_k, int64_t ld_dq_in,
                                  int64_t ld_dk_in, float eps, gbln_rope_pairing pairing,
                                  gbln_dtype io, gbln_dtype wt, gbln_stream_t stream);

/* Second pass: dwq[j] (+)= sum_p partial[p, j], dwk[j] (+)= sum_p partial[p, D + j], fixed order; [D] float32. */
gbln_status gbln_qk_norm_dw_finalize(const float* dw_partial, int64_t P, int32_t D, float* dwq,
                                     float* dwk, int accumulate, gbln_stream_t stream);

/*
 * gbln_rope_fwd_cache8 with the norms and position axes: q is normalised, rotated and
 * written, k normalised, rotated and quantised with v into their caches at the tokens'
 * slots.  rstd cancels out of k's codes, which are those of t = rotation of x * w (float32,
 * roundings written out), and goes into the scale: a = max(max |t|, 2^-100),
 * scale = (a * rstd) / qmax.  q_weight and k_weight both NULL: no norms (then with one
 * axis the same bits as gbln_rope_fwd_cache8).  Hq may be 0 (q, q_weight, q_out ignored);
 * Hk >= 1.  Slots, positions, aliasing and errors as there, D up to 512.
 */
gbln_status gbln_qk_norm_rope_fwd_cache8(const void* q, const void* k, const void* v,
                                         const void* q_weight, const void* k_weight, void* q_out,
                                         const int32_t* positions, int64_t ld_positions,
                                         int32_t n_axes, const uint8_t* axis, const float* cos_sin,
                                         int64_t max_pos, const int64_t* slots,
                                         const gbln_cache8* k_cache, const gbln_cache8* v_cache,
                                         int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                                         int64_t ld_q, int64_t ld_k, int64_t ld_v,
                                         int64_t ld_q_out, float eps, gbln_rope_pairing pairing,
                                         gbln_q8 fmt, gbln_dtype io, gbln_dtype wt,
                                         gbln_stream_t stream);

/*
 * Attention of the new tokens of a ragged batch over the paged cache (decode steps, drafts,
 * chunks of a prompt, whole prompts).  Sequence b has the rows cu_seqlens_q[b] ..
 * cu_seqlens_q[b + 1] - 1 of q, its last new tokens, whose keys and values are in the cache
 * already; kv_lens[b] tokens are cached in all, token j in slot j % page_size of page
 * page_table[b, j / page_size].  A row at position p (the last one at kv_lens[b] - 1) sees
 * the keys j <= p if causal, all if not, and of those with window > 0 only j > p - window:
 *   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j),  lse = log sum_j w_j
 * (k_j, v_j = code * scale).  Head h of q goes with K/V head h / (Hq / Hk).  A row that sees no
 * key gives zeros and lse -infinity.  Scores, weights, their sums and results are float32;
 * with bf16 rows and D 64, 96, 128 or 256 the weights times v's scales are rounded to 16 bits
 * for their products: to bf16 with many rows and D up to 128, else to fp16 relative to the power
 * of two above the scales of v that the row has met (11 bits; what is below 2^-38 of it becomes 0).
 * Keys that a row does not see have no part in it, whatever the cache holds there; pages that
 * no row of the sequence sees are not read (freed pages may hold any number in the table).
 * A row that sees a key with a scale of NaN is NaN.  What a row is that sees an E4M3 code of NaN
 * with another scale (no call here stores one) is not specified; other rows do not change.
 * cu_seqlens_q [B + 1], non-decreasing from 0, kv_lens [B], page_table [B, max_pages] int32,
 * read on the device (a captured call follows them); values beyond T or max_pages * page_size
 * are cut to it.  Rows behind cu_seqlens_q[B] are left as they are.  A page that is read and
 * lies outside the cache makes the rows that see it NaN and sets bit 4 of the error word.
 * q, out [T, Hq, D] io at t * ld + h * D; out may alias q exactly.  lse [T, Hq] float32 or NULL.
 * workspace: gbln_attn_cache8_workspace bytes (by the sizes and the device's SM count; 0: none
 * needed), 16-byte aligned, contents of no account; calls that may overlap need one each.
 * Bitwise reproducible for fixed sizes, lengths, alignment and GPU model.
 * Errors: INVALID_ARG for Hq not a multiple of Hk, D > 512, Hq * D above 2^24, T * Hq or
 * max_pages * page_size above 2^30, a scale that is not finite (or beyond 2e38), window < 0
 * and as gbln_cache8_read; WORKSPACE.
 */
int64_t gbln_attn_cache8_workspace(int64_t T, int32_t B, int32_t Hq, int32_t Hk, int32_t D,
                                   gbln_dtype io);
gbln_status gbln_attn_cache8(const void* q, const int32_t* cu_seqlens_q, const int32_t* kv_lens,
                             const int32_t* page_table, int64_t max_pages,
                             const gbln_cache8* k_cache, const gbln_cache8* v_cache, void* out,
                             float* lse, void* workspace, int64_t workspace_bytes, int64_t T,
                             int32_t B, int32_t Hq, int32_t Hk, int32_t D, int64_t ld_q,
                             int64_t ld_out, float scale, int32_t causal, int32_t window,
                             gbln_q8 fmt, gbln_dtype io, gbln_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GBLN_H */

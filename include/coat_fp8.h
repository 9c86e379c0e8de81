/*
 * coat_fp8.h -- C ABI of the MI355X (gfx950) FP8 AdamW optimizer step with
 * Dynamic Range Expansion (COAT, arXiv:2410.19313).
 *
 * Sources, cited by page and section:
 *   [P1] "COAT: Compressing Optimizer States and Activation for Memory-Efficient
 *        FP8 Training", paper review at xllm-io.github.io.  Section 三
 *        (技术架构) / 核心公式: quantizer equation "FP8量化", AdamW equation
 *        "AdamW优化器更新规则", expansion equations under "动态范围扩展"
 *        (f(x) = sign(x)|x|^k, R_f(X) = (R_X)^k, optimal k = log_{R_X} R_E4M3).
 *        Section 四 table: the optimizer state update is one fused kernel, and
 *        under FSDP each GPU handles its own shard with no cross-GPU range sync.
 *   [OCP] OCP 8-bit Floating Point Specification (OFP8): E4M3, bias 7,
 *        largest finite 448, smallest normal 2^-6, no infinities.
 *
 * State layout (one "moment" = m or v of one tensor of n elements, group size G):
 *   codes[n]            E4M3 codes, element i in byte i.  Sign in bit 7.
 *   scale[ceil(n/G)]    FP32: the group's max |x| before expansion.  0 marks an
 *                       all-zero group (k is then ignored).
 *   k[ceil(n/G)]        FP32: the group's expansion exponent, 0 < k <= 16.
 * Group j covers elements [j*G, min(n, (j+1)*G)).  Groups never cross tensors.
 * A value is stored as code = RNE_E4M3(448 * (|x|/scale)^k) with the sign of x
 * and read back as x = sign(code) * scale * (|code|/448)^(1/k).  Fresh state is
 * all-zero bytes (scale 0 everywhere).
 *
 * Conventions for every entry point:
 *   - Every array argument is DEVICE memory owned by the caller.  The library
 *     allocates nothing, keeps no per-call state, never synchronizes and never
 *     copies host<->device.  Host structs passed by pointer are read during the
 *     call only.
 *   - Work is enqueued on `stream` (0 = the null stream); results are valid
 *     once the caller synchronizes with that stream.
 *   - Arrays must not alias each other.  Codes, FP32 and BF16 element arrays
 *     must be 16-byte aligned; scale and k arrays 4-byte aligned.
 *   - Validation runs before anything is enqueued: any status other than
 *     COAT_ERR_HIP means nothing was launched and no buffer was touched.
 *     COAT_ERR_HIP means a launch failed (earlier launches of the same call may
 *     have run; the state is then undefined).
 *   - n == 0 is a successful no-op (pointers may then be NULL).
 *   - NaN or Inf in inputs is outside the contract.  Exactness (parity with the
 *     CPU reference to the documented tolerance) holds for groups whose
 *     dynamic range max|x| / min-nonzero|x| is at most 2^157.
 */
#ifndef COAT_FP8_H
#define COAT_FP8_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define COAT_FP8_ABI_VERSION 1

typedef enum coat_status {
  COAT_OK = 0,
  COAT_ERR_NULL_POINTER = 1,  /* a required pointer is NULL                 */
  COAT_ERR_INVALID_VALUE = 2, /* negative size, bad hyperparameter or step  */
  COAT_ERR_GROUP_SIZE = 3,    /* group_size not in {16, 32, 64, 128}         */
  COAT_ERR_MISALIGNED = 4,    /* an array violates the alignment rule above */
  COAT_ERR_HIP = 5            /* a HIP launch failed                        */
} coat_status_t;

/* One quantized moment (see "State layout"). */
typedef struct coat_fp8_state {
  uint8_t* codes;
  float* scale;
  float* k;
} coat_fp8_state_t;

/* One parameter tensor of an optimizer shard. */
typedef struct coat_adamw_tensor {
  float* w;              /* n FP32 master weights, updated in place      */
  const uint16_t* grad;  /* n BF16 gradient bit patterns, read only      */
  coat_fp8_state_t m;    /* first moment, updated in place               */
  coat_fp8_state_t v;    /* second moment, updated in place              */
  int64_t n;             /* number of elements, >= 0                     */
} coat_adamw_tensor_t;

typedef struct coat_adamw_hparams {
  float lr;           /* eta, finite                                       */
  float beta1;        /* in [0, 1)                                         */
  float beta2;        /* in [0, 1)                                         */
  float eps;          /* added to sqrt(v_hat), finite                      */
  float weight_decay; /* lambda, decoupled: w -= lr * lambda * w, finite   */
  int64_t step;       /* t of this update, >= 1; the caller increments it  */
  int32_t group_size; /* G in {16, 32, 64, 128}                            */
} coat_adamw_hparams_t;

/*
 * One fused AdamW step over a list of tensors ([P1] section 四: fused
 * optimizer kernel; [P1] 核心公式 AdamW, FP8量化 and 动态范围扩展).
 * Per group: dequantize m and v (invert the quantizer, then f), apply
 *   m_t = b1 m + (1-b1) g,  v_t = b2 v + (1-b2) g^2,
 *   w  <- w - lr ( (m_t/(1-b1^t)) / (sqrt(v_t/(1-b2^t)) + eps) + wd w ),
 * using the unquantized m_t and v_t, then store m_t and v_t again with a
 * fresh scale = max|x| and k = min(16, log2(448/2^-6) / log2(max|x|/min|x|))
 * (min over nonzero |x|; k = 16 when all nonzero magnitudes are equal).
 * The step is shard-local: it reads and writes only the given tensors.
 * Errors: COAT_ERR_NULL_POINTER (tensors/hp NULL, or a pointer of a tensor
 * with n > 0), COAT_ERR_INVALID_VALUE (num_tensors < 0, n < 0, step < 1,
 * beta outside [0,1), non-finite lr/eps/weight_decay), COAT_ERR_GROUP_SIZE,
 * COAT_ERR_MISALIGNED, COAT_ERR_HIP.
 */
coat_status_t coat_adamw_fp8_step(const coat_adamw_tensor_t* tensors,
                                  int32_t num_tensors,
                                  const coat_adamw_hparams_t* hp,
                                  hipStream_t stream);

/*
 * Expand and quantize an FP32 vector into a fresh state ([P1] 核心公式:
 * FP8量化 applied per group to f(X) with the group's optimal k).  Used to
 * convert FP32 optimizer states (e.g. a checkpoint) into FP8 state.
 * x: n FP32 values (read only).  out: codes[n], scale/k[ceil(n/G)] (written).
 * Errors: NULL_POINTER, INVALID_VALUE (n < 0), GROUP_SIZE, MISALIGNED, HIP.
 */
coat_status_t coat_fp8_expand_quantize(const float* x, int64_t n,
                                       int32_t group_size, coat_fp8_state_t out,
                                       hipStream_t stream);

/*
 * Dequantize and un-expand a state into FP32 ([P1] 核心公式: inverse of the
 * quantizer, then of f): x = sign(c) * scale * (|c|/448)^(1/k); a group with
 * scale 0 reads as zeros.  codes/scale/k read only; x[n] written.
 * Errors: NULL_POINTER, INVALID_VALUE (n < 0), GROUP_SIZE, MISALIGNED, HIP.
 */
coat_status_t coat_fp8_dequantize_expand(const uint8_t* codes,
                                         const float* scale, const float* k,
                                         int64_t n, int32_t group_size,
                                         float* x, hipStream_t stream);

/*
 * Plain OCP E4M3 conversion, element-wise ([OCP]; the rounding step the
 * quantizer ends in): codes[i] = round-to-nearest-even(x[i]), saturating at
 * +-448, sign kept (a negative value that rounds to zero gives 0x80).
 * Errors: NULL_POINTER, INVALID_VALUE (n < 0), MISALIGNED, HIP.
 */
coat_status_t coat_e4m3_encode(const float* x, int64_t n, uint8_t* codes,
                               hipStream_t stream);

/* Inverse of the above: x[i] = value of codes[i] (NaN for 0x7F / 0xFF). */
coat_status_t coat_e4m3_decode(const uint8_t* codes, int64_t n, float* x,
                               hipStream_t stream);

/*
 * Per-group FP8 quantization of an activation matrix, with its transpose
 * ([P1] section 三, 混合粒度激活量化: non-linear layers quantize per 1xG
 * group; Triton优化内核 / 非线性层优化: that kernel also writes the transposed
 * FP8 tensor the backward pass reads; [P1] 核心公式 FP8量化 with
 * S = max|X| / 448).  No range expansion (k = 1).
 *   x        rows x cols BF16 values (bit patterns), row-major (read only).
 *   codes    rows x cols E4M3 codes, row-major (written).
 *   scales   rows x (cols / group_size) FP32, row-major (written): group
 *            (i, j) covers x[i, j*G .. j*G+G-1] and stores S = max|x| / 448
 *            (IEEE division; 0 for an all-zero group).
 *   codes_t  cols x rows E4M3 codes, the transpose of `codes` (written), or
 *            NULL to skip it.
 * Each code is the E4M3 rounding (nearest, ties to even) of the exact
 * quotient 448 x / max|x|: the kernel forms it in FP32 with one residual
 * correction, which lands on every E4M3 value and midpoint exactly, and for
 * BF16 x no quotient lies close enough to a midpoint for the remaining error
 * to change a code.  Groups with max < 2^-100 are pre-scaled by 2^64.
 * -0 gives code 0x00, a negative x that rounds to zero 0x80, an all-zero
 * group codes 0.
 * cols must be a multiple of group_size.  x, codes and codes_t 16-byte
 * aligned, scales 4-byte aligned; writes into codes_t are 16, 8 or 4 bytes
 * wide when rows is a multiple of 16, 8 or 4, bytes otherwise.
 * Errors: NULL_POINTER (x/codes/scales NULL with rows, cols > 0),
 * INVALID_VALUE (rows or cols < 0, cols % group_size != 0, more than 2^31-1
 * tiles of 128 x 128), GROUP_SIZE, MISALIGNED, HIP.
 */
coat_status_t coat_fp8_quantize_act(const uint16_t* x, int64_t rows,
                                    int64_t cols, int32_t group_size,
                                    uint8_t* codes, float* scales,
                                    uint8_t* codes_t, hipStream_t stream);

/*
 * Group-scaled FP8 linear layer ([P1] section 三, Triton优化内核 / 线性层优化:
 * the GEMM output viewed as (BLOCK_M, BLOCK_N/G, G) with the max taken along
 * the last axis; section 四 table, 组缩放技术: a two-stage max reduction fused
 * into the producing operation; [P1] 核心公式 FP8量化 with S = max|X| / 448).
 *   C = s * A B^T with s = a_scale * b_scale, accumulated in FP32 on the
 *   matrix cores as c = A B^T, then each 1xG group of a row of C is
 *   quantized from C = fl(c s): S = max|C| / 448 (max|C| = fl(max|c| * |s|)
 *   exactly, rounding being monotone) and each code the E4M3 rounding of
 *   448 C / max|C|, formed as in coat_fp8_quantize_act but from the
 *   hardware reciprocal of max/512 (exact at every E4M3 value and midpoint;
 *   elsewhere a code can differ from the exact quotient's only for a
 *   quotient within about 2^-21 relative of a midpoint).  -0 -> 0x00, an all-zero group -> S = 0
 *   and codes 0; groups whose max lies below 2^-100 take the 2^64 pre-scale.
 *   a        M x K E4M3 codes, row-major (read only).
 *   b        N x K E4M3 codes, row-major (read only): the weight of a linear
 *            layer y = x W^T in its usual [out, in] layout.
 *   a_scale, b_scale  per-tensor scales, finite; their product s is
 *            rounded to FP32 once.
 *   codes    M x N E4M3 codes, row-major (written).
 *   scales   M x (N / group_size) FP32, row-major (written).
 *   c_f32    optional M x N FP32 fl(c s) before quantization (written), or NULL.
 * N and K must be multiples of 128, K <= 2^24; M is any size >= 0 (M or N
 * zero is a no-op; K zero gives C = 0, and a, b may then be NULL).  a, b,
 * codes and c_f32 16-byte aligned, scales 4-byte aligned.  NaN codes in a or
 * b are outside the contract.
 * Errors: NULL_POINTER, INVALID_VALUE (negative sizes, N or K not a multiple
 * of 128, K > 2^24, non-finite scales, grid too large), GROUP_SIZE,
 * MISALIGNED, HIP.
 */
coat_status_t coat_fp8_gemm_group_quant(const uint8_t* a, const uint8_t* b,
                                        float a_scale, float b_scale,
                                        int64_t M, int64_t N, int64_t K,
                                        int32_t group_size, uint8_t* codes,
                                        float* scales, float* c_f32,
                                        hipStream_t stream);

/*
 * The same FP8 GEMM with a plain epilogue: C = (a_scale * b_scale) * A B^T
 * rounded to BF16 (nearest even), c_bf16 M x N row-major (written).  It is
 * the reference point for the cost of the group-scaled epilogue above.
 * Arguments, layout and errors as above (no group_size).
 */
coat_status_t coat_fp8_gemm_bf16(const uint8_t* a, const uint8_t* b,
                                 float a_scale, float b_scale, int64_t M,
                                 int64_t N, int64_t K, uint16_t* c_bf16,
                                 hipStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Activation checkpoints: the operators between the linear layers, which keep
 * what their backward pass needs as E4M3 codes and read it there again ([P1]
 * section 三, 混合粒度激活量化: per 1xG group for non-linear layers, one scale
 * per tensor in front of linear layers).
 *
 * A checkpoint of a rows x cols matrix is what coat_fp8_quantize_act and
 * coat_fp8_gemm_group_quant write: codes rows x cols, scales
 * rows x (cols / group_size) with S = max|x| / 448, and stands for code * S.
 * Codes "under one scale" s stand for code * s; a value v is stored as the
 * E4M3 rounding of v * fl(1/s), saturating at +-448.  BF16 outputs and
 * gradients are rounded once, to nearest even, from FP32.
 *
 * The rules at the top hold, with these additions:
 *   - Optional arrays may be NULL.  Rows are contiguous except where a stride
 *     is an argument.
 *   - *_amax, if given, is raised to the largest magnitude (before the scale)
 *     of the FP32 values that were rounded to codes; it must hold a
 *     non-negative value before (0 to start a new maximum).  A NaN is not
 *     counted (its code is NaN).  The scales y_scale and h_scale are values of
 *     the call: a captured graph keeps those it was captured with, and a scale
 *     made from a maximum takes a copy to the host.
 *   - Gradients of weights are FP32 and sums over rows in a fixed order.
 *     accumulate != 0 adds them to what the array holds, else they overwrite
 *     it.  A weight gradient pointer may be NULL (a frozen weight).
 *   - workspace: device memory of at least the bytes that the *_workspace
 *     function gives for the same sizes, 16-byte aligned, its content neither
 *     read before it is written nor of use afterwards.  Calls, or replays of
 *     captured graphs, that share one must not overlap.
 *   - A NaN or infinity reaches no output outside its row (qk: its head,
 *     swiglu: its value) except the weight gradients, and in a checkpoint its
 *     group, whose codes are NaN and whose scale is not finite.
 */

/*
 * RMS norm of a residual stream with a checkpoint of its input:
 *   h = bf16(x + residual), or x without a residual,
 *   rstd = (mean(h^2) + eps)^-1/2,  y = h * rstd * weight.
 * cols is a multiple of group_size, at most 32768; squares are summed in FP32
 * (where that sum overflows rstd is 0).
 * Errors: NULL_POINTER (args, x, weight; neither y nor y_codes; residual
 * without residual_out or codes without scales, or the reverse),
 * INVALID_VALUE (sizes; eps not finite or below 2^-126; with y_codes, y_scale not
 * positive and finite or its reciprocal infinite; y_amax without y_codes),
 * GROUP_SIZE, MISALIGNED (16 bytes; scales, rstd and y_amax 4), HIP.
 */
typedef struct coat_rms_norm_args {
  const uint16_t* x;         /* rows x cols BF16                             */
  const uint16_t* residual;  /* rows x cols BF16, or NULL                    */
  const uint16_t* weight;    /* cols BF16                                    */
  uint16_t* residual_out;    /* h (written), with residual; may be residual  */
  uint16_t* y;               /* BF16 y (written), or NULL                    */
  uint8_t* y_codes;          /* y under one scale (written), or NULL         */
  float* y_amax;             /* optional, see above                          */
  uint8_t* codes;            /* checkpoint of h (written), or NULL           */
  float* scales;
  float* rstd;               /* rows FP32 (written), or NULL                 */
  int64_t rows, cols;
  float eps, y_scale;
  int32_t group_size;
} coat_rms_norm_args_t;

coat_status_t coat_fp8_rms_norm(const coat_rms_norm_args_t* args,
                                hipStream_t stream);

/*
 * Its gradient, with n = code * S * rstd and dn = dy * weight:
 *   dx = rstd * (dn - n * mean(dn * n)) (+ d_residual),
 *   dw = sum over rows of dy * n.
 * d_residual is the gradient that reaches residual_out from elsewhere; dx is
 * then the gradient of both x and residual.  dx must not be dy.
 * Errors: as above (codes, scales and rstd are required; workspace with dw;
 * INVALID_VALUE for a workspace that is too small and for dx == dy).
 */
typedef struct coat_rms_norm_bwd_args {
  const uint16_t* dy;          /* rows x cols BF16                           */
  const uint8_t* codes;        /* the checkpoint                             */
  const float* scales;
  const float* rstd;
  const uint16_t* weight;
  const uint16_t* d_residual;  /* rows x cols BF16, or NULL                  */
  uint16_t* dx;                /* rows x cols BF16 (written)                 */
  float* dw;                   /* cols FP32, or NULL                         */
  void* workspace;
  int64_t workspace_bytes;
  int64_t rows, cols;
  int32_t group_size, accumulate;
} coat_rms_norm_bwd_args_t;

coat_status_t coat_fp8_rms_norm_bwd(const coat_rms_norm_bwd_args_t* args,
                                    hipStream_t stream);

/* Bytes of workspace for that call, or -1 for sizes it refuses. */
int64_t coat_fp8_rms_norm_bwd_workspace(int64_t rows, int64_t cols);

/*
 * Gated activation h = gate * sigmoid(gate) * up.  A row of 2 * cols values
 * holds the gates, then the ups, as the packed projection leaves it.
 * Without gate_up the input is the checkpoint codes, scales (read), for
 * instance the output of coat_fp8_gemm_group_quant; with gate_up it is BF16,
 * and codes, scales, if given, are written as its checkpoint.
 * Exactly one of h and h_codes is given.  A sigmoid below 2^-126 is 0.
 * Errors: NULL_POINTER (args; no output; no input; codes without scales or
 * the reverse), INVALID_VALUE (sizes, cols not a multiple of group_size or
 * over 2^30, both outputs, h_scale as y_scale above, h_amax without h_codes),
 * GROUP_SIZE, MISALIGNED (16 bytes; scales and h_amax 4), HIP.
 */
typedef struct coat_swiglu_args {
  const uint16_t* gate_up;  /* rows x 2 cols BF16, or NULL                   */
  uint8_t* codes;           /* rows x 2 cols: the input, or the checkpoint   */
  float* scales;
  uint16_t* h;              /* rows x cols BF16 (written), or NULL           */
  uint8_t* h_codes;         /* h under one scale (written), or NULL          */
  float* h_amax;            /* optional, see above                           */
  int64_t rows, cols;
  float h_scale;
  int32_t group_size;
} coat_swiglu_args_t;

coat_status_t coat_fp8_swiglu(const coat_swiglu_args_t* args,
                              hipStream_t stream);

/*
 * Its gradient, with gate and up the checkpoint's values and s = sigmoid(gate):
 *   d_gate = dh * up * s * (1 + gate * (1 - s)),  d_up = dh * gate * s.
 * dh rows x cols BF16; d_gate_up rows x 2 cols BF16 (written), gates first.
 * Errors: as above.
 */
coat_status_t coat_fp8_swiglu_bwd(const uint16_t* dh, const uint8_t* codes,
                                  const float* scales, int64_t rows,
                                  int64_t cols, int32_t group_size,
                                  uint16_t* d_gate_up, hipStream_t stream);

/* Sizes that the two calls below share. */
typedef struct coat_qk_shape {
  int64_t tokens, table_rows;  /* table_rows: rows of cos and sin            */
  int32_t q_heads, k_heads;    /* each 0 to 65536                            */
  int32_t head_dim;            /* multiple of 16 and group_size, 16 to 256   */
  int32_t rot_dim;             /* rotated values: multiple of 16, <= head_dim */
  int32_t interleaved;         /* pairs (2j, 2j+1), else (j, j + rot_dim/2)  */
  int32_t group_size;
} coat_qk_shape_t;

/*
 * RMS norm of every query and key head and the position rotation:
 *   rstd = (mean over the head of x^2 + eps)^-1/2,  y = x * rstd * weight,
 * then pair j (a, b) of the first rot_dim values of y becomes
 *   (a cos_j - b sin_j, b cos_j + a sin_j),  cos and sin: row positions[token]
 * of the tables (table_rows x rot_dim/2 FP32).  The heads of a token are
 * contiguous (head h at h * head_dim); a stride counts the values from one
 * token to the next, so queries and keys may be parts of one packed
 * projection.  q_out may be q and k_out k, with equal strides.
 * The checkpoint and rstd hold the query heads of a token, then its key
 * heads: codes tokens x (q_heads + k_heads) x head_dim, scales
 * tokens x heads x head_dim / group_size, rstd tokens x heads.
 * A token whose position lies outside [0, table_rows) is padding: its
 * outputs, codes, scales and rstd are written as zero.
 * Errors: NULL_POINTER, INVALID_VALUE (sizes as above, a stride below a
 * token's values or not a multiple of 8, eps as above), GROUP_SIZE,
 * MISALIGNED (16 bytes; positions 8, scales and rstd 4), HIP.
 */
typedef struct coat_qk_norm_rope_args {
  coat_qk_shape_t shape;
  const uint16_t* q;        /* BF16 heads                                    */
  const uint16_t* k;
  int64_t q_stride, k_stride;
  const uint16_t* q_weight; /* head_dim BF16                                 */
  const uint16_t* k_weight;
  const float* cos;
  const float* sin;
  const int64_t* positions; /* tokens                                        */
  uint16_t* q_out;          /* BF16 heads (written)                          */
  uint16_t* k_out;
  int64_t q_out_stride, k_out_stride;
  uint8_t* codes;           /* checkpoint (written), or NULL                 */
  float* scales;
  float* rstd;              /* (written), or NULL                            */
  float eps;
} coat_qk_norm_rope_args_t;

coat_status_t coat_fp8_qk_norm_rope(const coat_qk_norm_rope_args_t* args,
                                    hipStream_t stream);

/*
 * Its gradient from the checkpoint: dy is d*_out rotated by minus the angle,
 * then as coat_fp8_rms_norm_bwd head by head; dq_weight and dk_weight sum
 * over tokens and heads.  Padding tokens get zero gradients and add nothing,
 * whatever their buffers hold.  dq may be dq_out and dk dk_out, with equal
 * strides.  Errors: as above (codes, scales and rstd are required; dq_weight
 * and dk_weight both or neither; workspace as above).
 */
typedef struct coat_qk_norm_rope_bwd_args {
  coat_qk_shape_t shape;
  const uint16_t* dq_out;   /* BF16 heads                                    */
  const uint16_t* dk_out;
  int64_t dq_out_stride, dk_out_stride;
  const uint8_t* codes;     /* the checkpoint                                */
  const float* scales;
  const float* rstd;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const float* cos;
  const float* sin;
  const int64_t* positions;
  uint16_t* dq;             /* BF16 heads (written)                          */
  uint16_t* dk;
  int64_t dq_stride, dk_stride;
  float* dq_weight;         /* head_dim FP32, or NULL                        */
  float* dk_weight;
  void* workspace;
  int64_t workspace_bytes;
  int32_t accumulate;
} coat_qk_norm_rope_bwd_args_t;

coat_status_t coat_fp8_qk_norm_rope_bwd(const coat_qk_norm_rope_bwd_args_t* args,
                                        hipStream_t stream);

/* Bytes of workspace for that call (heads: queries and keys), or -1. */
int64_t coat_fp8_qk_norm_rope_bwd_workspace(int64_t tokens, int64_t heads,
                                            int64_t head_dim);

/*
 * Weight gradient of a linear layer C = X W^T whose input X was kept in E4M3:
 *   dW[n][k] = sum over rows m of dy[m][n] * X[m][k],
 * X = code * S per group (x_scales) or code * x_scale (x_scales NULL),
 * accumulated in FP32 on the matrix cores.  Under one scale the codes' values
 * are exact in BF16 and x_scale multiplies the FP32 sum.  With group scales
 * code * S is rounded to BF16 for dw_bf16 (by at most 2^-8 of it); for dw_f32
 * it goes in as two BF16 values, which hold it to 2^-16, in twice the products.
 * N and K multiples of 16, K of group_size with x_scales; both at most 2^24.
 * Exactly one of dw_bf16 and dw_f32 is given; accumulate needs dw_f32.
 * M == 0 gives a zero gradient.  The workspace may be NULL when the workspace
 * function gives 0.
 * Errors: NULL_POINTER, INVALID_VALUE (sizes, x_scale not finite, dw_bf16
 * with dw_f32 or accumulate, a workspace that is too small), GROUP_SIZE,
 * MISALIGNED (16 bytes; x_scales 4), HIP.
 */
typedef struct coat_weight_grad_args {
  const uint16_t* dy;      /* M x N BF16                                     */
  const uint8_t* x_codes;  /* M x K                                          */
  const float* x_scales;   /* M x K/group_size, or NULL                      */
  uint16_t* dw_bf16;       /* N x K BF16 (written), or NULL                  */
  float* dw_f32;           /* N x K FP32 (written or added to), or NULL      */
  void* workspace;
  int64_t workspace_bytes;
  int64_t M, N, K;
  float x_scale;
  int32_t group_size, accumulate;
} coat_weight_grad_args_t;

coat_status_t coat_fp8_weight_grad(const coat_weight_grad_args_t* args,
                                   hipStream_t stream);

/* Bytes of workspace for that call, or -1 for sizes it refuses. */
int64_t coat_fp8_weight_grad_workspace(int64_t M, int64_t N, int64_t K);

/*
 * ---------------------------------------------------------------------------
 * The vocabulary: the operators at the two ends of a model, which read a
 * vocab x cols matrix (one matrix where the two are tied) and whose gradients
 * the optimizer step above takes.
 *
 * Matrices are BF16, or E4M3 codes under one scale (code * scale).  A token or
 * target outside [0, vocab) is padding: its rows of outputs are zero, what its
 * rows of inputs hold (NaN included) reaches nothing, and it adds to no
 * gradient.  vocab at most 2^22, cols 65536, rows 2^23; rows * cols at most
 * 2^33 and vocab * cols 2^34.  Gradients of the matrix are BF16 (written) or
 * FP32 (written or, with accumulate, added to); sums are FP32 and their order
 * is fixed by the sizes and inputs, no float is added by an atomic.
 */

/*
 * Embedding lookup: out[r] = bf16(scale * table[tokens[r]]).
 * scale * table_scale is rounded to FP32 once.  cols a multiple of 16.
 * Errors: NULL_POINTER (args; tokens, out, table with vocab > 0),
 * INVALID_VALUE (sizes, both tables, a scale not finite), MISALIGNED (16
 * bytes; tokens 8), HIP.
 */
typedef struct coat_embedding_args {
  const uint16_t* table;       /* vocab x cols BF16, or NULL                 */
  const uint8_t* table_codes;  /* vocab x cols E4M3 under table_scale        */
  const int64_t* tokens;       /* rows                                       */
  uint16_t* out;               /* rows x cols BF16 (written)                 */
  int64_t rows, vocab, cols;
  float table_scale, scale;    /* table_scale: 1 for a BF16 table            */
} coat_embedding_args_t;

coat_status_t coat_fp8_embedding(const coat_embedding_args_t* args,
                                 hipStream_t stream);

/*
 * Its gradient: dw[v] = scale * sum of dy[r] over the rows with tokens[r] = v,
 * summed in FP32 in the rows' order (32 rows of a token to a partial sum);
 * rows of tokens that do not occur are zero, or left as they are with
 * accumulate.  Errors: as above (workspace with rows > 0; INVALID_VALUE for
 * dw_bf16 with dw_f32 or accumulate and for a workspace that is too small).
 */
typedef struct coat_embedding_bwd_args {
  const uint16_t* dy;      /* rows x cols BF16                               */
  const int64_t* tokens;   /* rows                                           */
  uint16_t* dw_bf16;       /* vocab x cols BF16 (written), or NULL           */
  float* dw_f32;           /* vocab x cols FP32, or NULL                     */
  void* workspace;
  int64_t workspace_bytes;
  int64_t rows, vocab, cols;
  float scale;
  int32_t accumulate;
} coat_embedding_bwd_args_t;

coat_status_t coat_fp8_embedding_bwd(const coat_embedding_bwd_args_t* args,
                                     hipStream_t stream);

/* Bytes of workspace for that call, or -1 for sizes it refuses. */
int64_t coat_fp8_embedding_bwd_workspace(int64_t rows, int64_t vocab,
                                         int64_t cols);

/*
 * Softmax cross entropy of hidden states x against a vocabulary, from the
 * output projection's weights, without the logits in memory:
 *   l[v] = logit_scale * x . w[v],  lse = log sum over v of exp(l[v]),
 *   loss = lse - l[target] + z_loss * lse^2.
 * x and weight are both BF16 or both E4M3 (x_scale, weight_scale: 1 for
 * BF16); products are summed in FP32 on the matrix cores (which cut each of
 * eight neighbouring products of codes 13 bits below the largest; the target's
 * logit of codes is formed in FP32 instead), the exponentials in FP32.  cols is a
 * multiple of 64 for BF16, of 128 for E4M3, and ceil(rows / 256) *
 * ceil(vocab / 256) at most 2^22.  Rows without a target get loss
 * 0 and lse 0.  A NaN or infinity in a row of x reaches that row's results
 * alone.
 * Errors: NULL_POINTER (args; x, weight, targets, loss, workspace),
 * INVALID_VALUE (sizes; BF16 with E4M3; a scale, or the product of
 * logit_scale with one or both others, that is not positive, finite and at
 * least 2^-126; log2(e) times the product of all three not finite; z_loss not
 * finite; a workspace that is too small; vocab or
 * cols 0 with rows), MISALIGNED (16 bytes; targets 8, loss and lse 4), HIP.
 */
typedef struct coat_cross_entropy_args {
  const uint16_t* x;            /* rows x cols BF16, or NULL                 */
  const uint8_t* x_codes;       /* rows x cols E4M3, or NULL                 */
  const uint16_t* weight;       /* vocab x cols BF16, or NULL                */
  const uint8_t* weight_codes;  /* vocab x cols E4M3, or NULL                */
  const int64_t* targets;       /* rows                                      */
  float* loss;                  /* rows FP32 (written)                       */
  float* lse;                   /* rows FP32 (written), or NULL              */
  void* workspace;
  int64_t workspace_bytes;
  int64_t rows, vocab, cols;
  float x_scale, weight_scale, logit_scale, z_loss;
} coat_cross_entropy_args_t;

coat_status_t coat_fp8_cross_entropy(const coat_cross_entropy_args_t* args,
                                     hipStream_t stream);

/* Bytes of workspace for that call, or -1 for sizes it refuses. */
int64_t coat_fp8_cross_entropy_workspace(int64_t rows, int64_t vocab,
                                         int64_t cols);

/*
 * Its gradients, with d = d_loss of the row and the lse that the call above
 * wrote:
 *   g[v] = d ((1 + 2 z_loss lse) exp(l[v] - lse) - [v = target]),
 *   dx = logit_scale * g W,  dw = logit_scale * g^T x.
 * The logits are computed again as above, a piece of the vocabulary at a time:
 * as few pieces as the workspace holds (the FP32 sums of dx depend on their
 * number).
 * g, divided by the largest |d|, is rounded to BF16 (by at most 2^-8 of it)
 * for dx and a BF16 dw; an FP32 dw takes it in two BF16 parts, which hold it
 * to 2^-16, in twice the products, and so do both of up to 64 rows.  The
 * largest |d| times logit_scale and weight_scale (for dx) or x_scale (for dw)
 * is formed in FP32.  dx or the dw pointers may be NULL.
 * Errors: as above (lse and d_loss required; neither dx nor dw is
 * NULL_POINTER; dw_bf16 with dw_f32 or accumulate is INVALID_VALUE).
 */
typedef struct coat_cross_entropy_bwd_args {
  const float* d_loss;          /* rows FP32                                 */
  const uint16_t* x;            /* as above                                  */
  const uint8_t* x_codes;
  const uint16_t* weight;
  const uint8_t* weight_codes;
  const int64_t* targets;
  const float* lse;             /* rows FP32                                 */
  uint16_t* dx;                 /* rows x cols BF16 (written), or NULL       */
  uint16_t* dw_bf16;            /* vocab x cols BF16 (written), or NULL      */
  float* dw_f32;                /* vocab x cols FP32, or NULL                */
  void* workspace;
  int64_t workspace_bytes;
  int64_t rows, vocab, cols;
  float x_scale, weight_scale, logit_scale, z_loss;
  int32_t accumulate;
} coat_cross_entropy_bwd_args_t;

coat_status_t coat_fp8_cross_entropy_bwd(
    const coat_cross_entropy_bwd_args_t* args, hipStream_t stream);

/*
 * Bytes of workspace for that call in no more pieces of the vocabulary than
 * `piece` rows each make (rounded up to a multiple of 256), or -1 for sizes it
 * refuses.  vocab gives what one piece takes, 1 the least that any number of
 * them takes; a larger `piece` never gives less.  codes: x and weight are E4M3;
 * f32: dw is FP32.
 */
int64_t coat_fp8_cross_entropy_bwd_workspace(int64_t rows, int64_t vocab,
                                             int64_t cols, int64_t piece,
                                             int32_t codes, int32_t f32);

/* Static, NUL-terminated description of a status code. */
const char* coat_status_string(coat_status_t status);

/* HIP error string of the last COAT_ERR_HIP returned on the calling thread
 * (empty string if none). */
const char* coat_last_hip_error(void);

/* COAT_FP8_ABI_VERSION of the loaded library. */
int32_t coat_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* COAT_FP8_H */

/*
 * moe_train.h - C interface of the operators that train the dense branch of the hybrid
 * feed-forward block (see moe_ffn.h) on NVIDIA B200 (sm_100a): the norm before and after
 * the dense MLP, the gated MLP itself, each with its backward pass, and the 8-bit
 * checkpoints of activations that the backward passes read.
 *
 * The conventions of moe_ffn.h hold here too: row-major device memory owned by the caller,
 * work enqueued on `stream` only, argument errors found on the host before anything is
 * launched, nothing allocated, nothing thrown, bounded device waits, deterministic results.
 * In addition:
 *   - Activations are described by moe_act_t and may have rows `ld` elements apart, ld >=
 *     their columns.  The gaps between rows are neither read for results nor written.
 *   - Every tensor pointer is 16-byte aligned, scales excepted (any alignment).
 *   - Outputs must not overlap inputs or one another, unless a function says otherwise.
 *   - 0 <= T <= 2^31 - 512 rows.  T = 0 computes nothing, but weight gradients that are not
 *     accumulated are set to zero.
 *   - A workspace is 256-byte aligned and zeroed once before its first use; its first word
 *     is the status word that moe_check_device_status() reads.  It serves any calls in turn
 *     that it is large enough for, those of moe_ffn.h too.  Calls whose kernels may overlap
 *     on the GPU (other streams, other captured graphs) need workspaces of their own.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_F_BF16 = 0,
  MOE_F_F16 = 1,
  MOE_F_F32 = 2,
  MOE_F_INT8 = 3, /* 8-bit checkpoint, int8 codes */
  MOE_F_E4M3 = 4  /* 8-bit checkpoint, E4M3 codes */
} moe_format_t;

/* An activation [rows][cols].
 *
 * 8-bit checkpoints hold the columns in groups of 32 consecutive values (the last group of
 * a row may be shorter), each with a power-of-two scale:
 *   s = 2^k, the smallest with max|v| <= Q s and k >= -126, Q = 127 (int8) or 448 (E4M3);
 *   codes = v / s rounded to nearest even (exact division; never saturates);
 *   scale byte = k + 127, an all-zero group having byte 1.
 * A group that holds an infinity or NaN gets scale byte 255 and codes 0, and reads back as
 * NaN throughout.  Since s is a power of two, code * s is exact in bf16 (and in fp16 within
 * its normal range): reading a checkpoint adds no second rounding.
 *
 * code * s may lie a rounding above what a format holds.  Read back in 16 bits, values past
 * the format's largest finite one become that one, so a finite 16-bit activation never reads
 * back as an infinity (fp16: 65504 is kept as 64 * 2^10 and reads back as 65504).  In fp32,
 * as F32 and where the backward passes compute, kept values of at least 2^128 (1 - 2^-7) for
 * int8 and 2^128 (1 - 2^-5) for E4M3 are 2^128: infinity. */
typedef struct {
  void* data;      /* elements of `format`, row r at element r * ld */
  uint8_t* scales; /* 8-bit formats: [rows][ceil(cols / 32)] scale bytes; else NULL */
  int64_t ld;      /* elements from one row to the next */
  int32_t format;  /* moe_format_t */
} moe_act_t;

/* Writes the 8-bit checkpoint `dst` of `src` (BF16, F16 or F32), and reads the checkpoint
 * `src` back into `dst` (BF16, F16 or F32, rounded to nearest even; see above for values past
 * the largest).
 * rows >= 0, 1 <= cols <= 65536, rows * cols < 2^46. */
moe_status_t moe_act_encode(int64_t rows, int32_t cols, const moe_act_t* src,
                            const moe_act_t* dst, void* stream);
moe_status_t moe_act_decode(int64_t rows, int32_t cols, const moe_act_t* src,
                            const moe_act_t* dst, void* stream);

/* Row norms, statistics and sums in fp32.
 *   MOE_NORM_RMS:   rstd = 1 / sqrt(mean(x^2) + eps),        z = x rstd
 *   MOE_NORM_LAYER: rstd = 1 / sqrt(mean((x-mu)^2) + eps),   z = (x - mu) rstd
 *   y = z * gain + bias   (gain NULL: 1; bias, LAYER only, NULL: 0)
 * 1 <= cols <= 16384. */
typedef enum { MOE_NORM_RMS = 0, MOE_NORM_LAYER = 1 } moe_norm_kind_t;

typedef struct {
  int32_t kind;         /* moe_norm_kind_t */
  int32_t cols;
  float eps;            /* > 0 */
  int32_t format;       /* of x, y, dy and dx: BF16, F16 or F32 */
  int32_t param_format; /* of gain and bias: BF16, F16 or F32 */
} moe_norm_config_t;

/* y, the statistics the backward pass needs, and on request (`kept` not NULL) the 8-bit
 * checkpoint of x, written from the same pass over x.
 *   mean [T] fp32 (LAYER; NULL for RMS), rstd [T] fp32.  y may be x itself (same ld). */
moe_status_t moe_norm_forward(const moe_norm_config_t* cfg, int32_t T, const moe_act_t* x,
                              const void* gain, const void* bias, const moe_act_t* y,
                              float* mean, float* rstd, const moe_act_t* kept, void* stream);

/* The gradients, with a = dy * gain and z from x and the forward pass's statistics:
 *   dx     = rstd (a - z mean(a z) - mean(a))     (the last term for LAYER only)
 *   d_gain = sum over rows of dy z,  d_bias = sum over rows of dy,   fp32 [cols]
 * x: what the forward pass normalised, or its 8-bit checkpoint.  d_gain and d_bias may be
 * NULL (not computed; d_bias LAYER only); with accumulate != 0 they are added to what the
 * buffers hold.  dx may be dy itself (same ld).
 * ws: moe_norm_workspace_size(cfg, T) bytes (a host function; 0 if cfg is invalid). */
size_t moe_norm_workspace_size(const moe_norm_config_t* cfg, int32_t T);
moe_status_t moe_norm_backward(const moe_norm_config_t* cfg, int32_t T, const moe_act_t* x,
                               const void* gain, const float* mean, const float* rstd,
                               const moe_act_t* dy, const moe_act_t* dx, float* d_gain,
                               float* d_bias, int32_t accumulate, void* ws, size_t ws_bytes,
                               void* stream);

/* The gated MLP: g, u = x Wg^T, x Wu^T;  h = act(g) * u;  y = h Wd^T, with fp32 sums.
 *   act = gelu_tanh (the block's) or silu (g / (1 + exp(-g))).
 *   w_gate_up [2D][H] (gate rows, then up rows), w_down [H][D], as in moe_block_weights_t.
 * H and D: multiples of 8, 8..16384; all 16-bit tensors of one format, and every ld a
 * multiple of 8. */
typedef enum { MOE_ACT_GELU_TANH = 0, MOE_ACT_SILU = 1 } moe_activation_t;

typedef struct {
  int32_t hidden; /* H */
  int32_t inter;  /* D */
  int32_t act;    /* moe_activation_t */
  int32_t format; /* BF16 or F16 */
} moe_mlp_config_t;

/* Bytes of workspace for either pass over T rows (0 if cfg is invalid).  Host function. */
size_t moe_mlp_workspace_size(const moe_mlp_config_t* cfg, int32_t T);

/* x [T][H] -> y [T][H].  kept_gu: NULL, or [T][2D] that receives g (columns 0..D-1) and u
 * (columns D..2D-1) for the backward pass, in cfg's format or as 8-bit checkpoints written
 * from the fp32 sums.  The two halves are checkpoints of their own: scales
 * [T][2 ceil(D / 32)], the gate's groups first.  h is rounded to the 16-bit format between
 * the two products (the tensor cores' operand type). */
moe_status_t moe_mlp_forward(const moe_mlp_config_t* cfg, int32_t T, const moe_act_t* x,
                             const void* w_gate_up, const void* w_down, const moe_act_t* y,
                             const moe_act_t* kept_gu, void* ws, size_t ws_bytes, void* stream);

/* With dh = dy Wd, dg = dh u act'(g), du = dh act(g), h = act(g) u (recomputed from g, u):
 *   dx = [dg du] [Wg; Wu],   dw_gate_up = [dg du]^T x,   dw_down = dy^T h.
 * x [T][H] and gu [T][2D]: as kept, in cfg's format or 8 bits each.  dx, dw_gate_up and
 * dw_down may be NULL (not computed).  The weight gradients are contiguous, in grad_format
 * (cfg's format or F32); accumulate != 0 adds to what they hold (one rounding).  dg, du and
 * h are rounded to the 16-bit format between the products. */
moe_status_t moe_mlp_backward(const moe_mlp_config_t* cfg, int32_t T, const moe_act_t* x,
                              const moe_act_t* gu, const void* w_gate_up, const void* w_down,
                              const moe_act_t* dy, const moe_act_t* dx, void* dw_gate_up,
                              void* dw_down, int32_t grad_format, int32_t accumulate, void* ws,
                              size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */

/*
 * conv_seq.h — C ABI of the sequence operators: the causal depthwise
 * convolution along time, the selective state-space scan and the
 * root-mean-square norm, for prompts, training and single tokens. Around
 * them the pointwise (1x1) convolutions of conv_igemm.h are the projections
 * of a token-mixing layer.
 *
 * Conventions shared by every entry point
 *  - Tensors are channels-last: [n][l][c] with the channels contiguous. A
 *    seq_tensor gives its strides over sequences and tokens in elements, so a
 *    part of a wider buffer (one half of a projection's output) is taken and
 *    written in place. Input strides are >= 0 (0 repeats a row or a token; the
 *    stride along a single sequence or token is not used);
 *    an output's rows may not overlap: stride_l >= c and
 *    stride_n >= (l-1) stride_l + c, or the same with n and l exchanged.
 *    Pointers are aligned to their element; 16-byte aligned pointers and
 *    strides select the vector kernels, others run element by element. (The
 *    scan's states and their gradients have to be 16-byte aligned where s is a
 *    multiple of 4, its checkpoints and the workspaces always.)
 *  - States, weights and parameters are dense. All memory and the stream belong
 *    to the current device.
 *  - Types: `dtype` (CONV_F32, CONV_BF16 or CONV_F16) is the type of the token
 *    tensors. All arithmetic, states of the scan and sums are in fp32; each
 *    output is rounded once (to nearest even) into its type. Gradients of
 *    parameters are fp32.
 *  - `lengths` ([n] int32 on the device, or NULL: all l tokens) is the number
 *    of tokens of each sequence, taken as 0 when negative and as l when above
 *    l. Tokens at and past the length are not used, whatever they hold (NaN
 *    included): outputs and gradients there are 0, and the final state is the
 *    one after the last token inside. A length of 0 leaves the state as it was.
 *  - Nothing is allocated, nothing synchronises; kernels are enqueued on
 *    `stream` (a cudaStream_t; NULL = the legacy default stream), and every
 *    call can be captured into a CUDA graph. The caller owns all buffers; a
 *    workspace needs no clearing. No atomics on results: a call repeated on
 *    the same inputs gives the same bits.
 *  - Errors: every argument is checked before the first launch, so a status
 *    other than CONV_OK and CONV_ERR_CUDA means nothing was enqueued. A call
 *    without elements (n, l or c of 0, where allowed) enqueues what its other
 *    outputs need and returns CONV_OK.
 *  - An output must not overlap another tensor of the call, except where a
 *    call says that it updates one in place.
 */
#ifndef CONV_SEQ_H
#define CONV_SEQ_H

#include "conv_igemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A view of tokens: element (i, t, c) is data[i stride_n + t stride_l + c]. */
typedef struct seq_tensor {
  void* data;
  int64_t stride_n, stride_l;
} seq_tensor;

/* ---------------------------------------------------------------- causal convolution
 *
 *   v[t][c] = bias[c] + sum_{j < width} w[c][j] x[t - (width-1) + j][c]
 *   y = v, or silu(v) = v / (1 + exp(-v)) when silu is set
 *
 * x at times -(width-1) .. -1 comes from `state` ([n][width-1][c], row j is
 * time j - (width-1)), or is 0 when state is NULL. 1 <= width <= 4. */
typedef struct seq_conv_args {
  int64_t n, l, c, width;
  int32_t dtype;          /* x, y, dy, dx and the states */
  int32_t w_dtype;        /* w and bias: dtype or CONV_F32 */
  int32_t silu;           /* 0 or 1 */
  int32_t reserved;       /* 0 */
  seq_tensor x;           /* [n][l][c] */
  seq_tensor y;           /* forward, step: output */
  seq_tensor dy;          /* backward: gradient of y */
  seq_tensor dx;          /* backward: output */
  const void* w;          /* [c][width] */
  const void* bias;       /* [c] or NULL */
  const void* state;      /* [n][width-1][c] or NULL */
  void* state_out;        /* forward: the state after the last token, or NULL; may be `state` itself */
  const int32_t* lengths; /* [n] or NULL */
  const void* dstate_out; /* backward: gradient of state_out, or NULL (0) */
  void* dstate;           /* backward: gradient of state, or NULL */
  float* dw;              /* backward: [c][width] */
  float* db;              /* backward: [c], or NULL */
  const int32_t* slots;   /* step: [n] or NULL */
  int64_t n_slots;        /* step: states in the pool */
  void* ws;               /* backward */
  uint64_t ws_bytes;
} seq_conv_args;

/* y (and state_out) from x, w, bias, state. */
conv_status seq_conv_fwd(const seq_conv_args* a, void* stream);

/* Gradients of seq_conv_fwd: dx, dw, db, dstate from x, w, bias, state, dy,
 * dstate_out. dw sums over sequences and tokens in a fixed order, through
 * partial sums in ws (seq_conv_workspace_bytes). */
conv_status seq_conv_bwd(const seq_conv_args* a, void* stream);
conv_status seq_conv_workspace_bytes(int64_t n, int64_t l, int64_t c, int64_t width, uint64_t* bytes);

/* One token for each sequence (l = 1; stride_l is not used): y from x and the
 * state, which moves on by the token in place. state_out is a pool
 * [n_slots][width-1][c]; sequence i uses entry slots[i] (slots NULL: entry i,
 * n_slots >= n). A slot outside 0 .. n_slots-1 marks an empty row: no state is
 * touched and y is 0. Two rows must not share a slot. */
conv_status seq_conv_step(const seq_conv_args* a, void* stream);

/* ---------------------------------------------------------------- selective scan
 *
 *   delta[t][c] = dt[t][c] + dt_bias[c], or softplus of it
 *   h[t][c][k]  = exp(delta A[c][k]) h[t-1][c][k] + delta x[t][c] B[t][g(c)][k]
 *   y[t][c]     = (sum_{k < s} C[t][g(c)][k] h[t][c][k] + D[c] x[t][c]) * silu(z[t][c])
 *
 * with s states a channel (1 <= s <= 64), B and C shared by the c/g channels
 * of a group (g divides c; channel i is in group i / (c/g)), h[-1] = state or
 * 0, and the factor silu(z) and the term D x left out where z or D is NULL. */
typedef struct seq_scan_args {
  int64_t n, l, c, s, g;
  int32_t dtype;          /* x, dt, b, c, z, y and their gradients */
  int32_t softplus;       /* 0 or 1 */
  seq_tensor x, dt, z;    /* [n][l][c]; z.data may be NULL */
  seq_tensor b, cc;       /* [n][l][g][s], g and s dense */
  seq_tensor y;           /* forward, step: output */
  const float* A;         /* [c][s] */
  const float* D;         /* [c] or NULL */
  const float* dt_bias;   /* [c] or NULL */
  const float* state;     /* [n][c][s] or NULL */
  float* state_out;       /* forward: the state after the last token or NULL; may be `state` itself */
  const int32_t* lengths; /* [n] or NULL */
  float* checkpoints;     /* forward: output or NULL; backward: what the forward wrote; 16-byte aligned */
  seq_tensor dy;          /* backward: gradient of y */
  seq_tensor dx, ddt, dz; /* backward: outputs; dz with z only */
  seq_tensor db, dc;      /* backward: outputs [n][l][g][s] */
  float* dA;              /* backward: [c][s] */
  float* dD;              /* backward: [c], with D only, or NULL */
  float* ddt_bias;        /* backward: [c], with dt_bias only, or NULL */
  const float* dstate_out;/* backward: gradient of state_out or NULL (0) */
  float* dstate;          /* backward: gradient of state, or NULL */
  const int32_t* slots;   /* step: [n] or NULL */
  int64_t n_slots;        /* step: states in the pool */
  void* ws;               /* forward, backward */
  uint64_t ws_bytes;
} seq_scan_args;

/* y (and state_out, checkpoints) over a prompt. Where sequences times
 * channels are too few to fill the GPU the time axis is cut into segments,
 * whose entry states go through ws. checkpoints keeps the states that the
 * backward pass starts its recomputation from, in a layout of the library's. */
conv_status seq_scan_fwd(const seq_scan_args* a, void* stream);

/* Gradients of seq_scan_fwd with the same arguments, from the checkpoints it
 * wrote. Sums over tokens, sequences and a group's channels run in a fixed
 * order, through partial sums in ws. */
conv_status seq_scan_bwd(const seq_scan_args* a, void* stream);

/* Bytes of the workspace for sequences of this shape on a GPU with sm_count
 * SMs, or on the current device; and of the checkpoints. */
conv_status seq_scan_workspace_bytes_for(int64_t n, int64_t l, int64_t c, int64_t s, int64_t g, int32_t backward,
                                         int32_t sm_count, uint64_t* bytes);
conv_status seq_scan_workspace_bytes(int64_t n, int64_t l, int64_t c, int64_t s, int64_t g, int32_t backward,
                                     uint64_t* bytes);
conv_status seq_scan_checkpoint_bytes(int64_t n, int64_t l, int64_t c, int64_t s, uint64_t* bytes);

/* One token for each sequence (l = 1): y from the token and the state, which
 * moves on in place. state_out is a pool [n_slots][c][s]; slots as for
 * seq_conv_step. */
conv_status seq_scan_step(const seq_scan_args* a, void* stream);

/* ---------------------------------------------------------------- root-mean-square norm
 *
 *   r = x + residual (rounded into dtype; x itself without a residual)
 *   y[i][c] = r[i][c] rstd[i] w[c],   rstd[i] = 1 / sqrt(mean_c r[i][c]^2 + eps)
 *
 * y in dtype, or in 8 bits (e4m3) with a scale for every row (group 0) or for
 * every `group` columns of a row (32, 64 or 128; the last group may be
 * shorter): scale = max |y| / 448 over the group, q = y / scale. A group whose
 * maximum is not a number, or so small that the scale would round to 0, has scale 1. */
typedef struct seq_norm_args {
  int64_t n, c;           /* rows, columns */
  int32_t dtype;          /* x, residual, r, y, dy, dr, dx */
  int32_t w_dtype;        /* w: dtype or CONV_F32 */
  int32_t out8;           /* 1: y is e4m3 and scale is written */
  int32_t group;          /* 0, 32, 64 or 128 (out8 only) */
  float eps;              /* >= 0 */
  int32_t reserved;       /* 0 */
  /* Rows [n][c]; stride_l is not used. */
  seq_tensor x;           /* forward */
  seq_tensor residual;    /* forward; data may be NULL */
  seq_tensor y;           /* forward: output */
  seq_tensor r;           /* forward: output, data may be NULL (may be x or residual itself); backward: input (x without
                             a residual) */
  seq_tensor dy;          /* backward: gradient of y */
  seq_tensor dr;          /* backward: gradient of r from elsewhere; data may be NULL */
  seq_tensor dx;          /* backward: gradient of x and of residual; may be dr itself */
  const void* w;          /* [c] */
  float* scale;           /* forward: [n][ceil(c / group)] ([n] for group 0) when out8 */
  float* rstd;            /* forward: output [n] or NULL; backward: input */
  float* dw;              /* backward: [c] */
  void* ws;               /* backward */
  uint64_t ws_bytes;
} seq_norm_args;

conv_status seq_norm_fwd(const seq_norm_args* a, void* stream);
conv_status seq_norm_bwd(const seq_norm_args* a, void* stream);
conv_status seq_norm_workspace_bytes(int64_t n, int64_t c, uint64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* CONV_SEQ_H */

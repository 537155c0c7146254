/*
 * retention_block.h — C ABI of the operators around retention in a gated
 * recurrent block (gfx950 / MI355X): a linear recurrence whose decay is
 * computed per token and channel (retention's decay is fixed per head), and
 * the norms before and after the block's mixer with their gradients.
 *
 * Conventions are those of retention.h (status codes, element types RET_F32
 * and RET_BF16, streams, ownership: the library allocates nothing, and no
 * entry point throws or synchronises), with these additions:
 *   - A tensor of activations is a retention_view_t: [B, H, N, d] with the
 *     last dimension contiguous and the strides of the others given in
 *     elements (>= 0), so that a slice of a larger projection or a
 *     token-major tensor is taken in place. The data must be aligned to its
 *     element. A stride of an input may be 0 (a broadcast input); an output
 *     must not have two elements in one place. The stride of a dimension of
 *     size 1 is not read.
 *   - An output must not share bytes with an input or another output; the
 *     whole range a view spans counts, unless the two are columns of one larger
 *     tensor side by side (rows, or tokens of heads that follow one another, at
 *     the same distance). Such calls are refused with
 *     RET_ERR_INVALID_ARG, as are null pointers where a tensor is required,
 *     sizes <= 0 and misaligned data; RET_ERR_UNSUPPORTED: sizes beyond the
 *     limits stated at each function.
 *   - Sums, statistics and states are held in fp32; results in the element
 *     type are rounded once, to nearest even. The last h of a sequence is its
 *     final state, rounded.
 *   - Results do not depend on timing: calls with the same arguments on the
 *     same data give the same bits (no floating-point atomics).
 */
#ifndef RETENTION_BLOCK_H
#define RETENTION_BLOCK_H

#include <stddef.h>

#include "retention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Widest row of retention_residual_norm. */
#define RETENTION_MAX_MODEL_DIM 16384

typedef struct retention_view_t {
  void* data; /* device; never written through an input's view */
  long long stride_b, stride_h, stride_n; /* in elements */
} retention_view_t;

/*
 * Added to the dtype of retention_gated_recurrence and its backward
 * (RET_BF16 | RETENTION_H_F32): h alone is fp32. The backward reads h_{t-1}
 * from h, so with this grad_gate is formed without h's rounding to bf16, which
 * otherwise adds a second rounding of its size to it (error against 64 bits,
 * 2-norm, log form with memories of 2 to 500 tokens: 1.7e-3 against 2.3e-3).
 */
#define RETENTION_H_F32 0x100

/* How a gate value g becomes the decay a of a token and channel. */
enum retention_gate_form {
  RET_GATE_SIGMOID = 0, /* a = 1 / (1 + e^-g), the input weighted by 1 - a */
  RET_GATE_LOG = 1      /* a = e^g (g <= 0 for a decay), the input as it is */
};

/*
 * Gated linear recurrence over sequences, per channel:
 *   RET_GATE_SIGMOID:  h_t = a_t h_{t-1} + (1 - a_t) x_t
 *   RET_GATE_LOG:      h_t = a_t h_{t-1} + x_t
 * with h_{-1} = state_in (fp32 [sequences, H, d], NULL: zeros). A gate of -inf
 * (a = 0) starts the state anew at that token whatever it holds before, NaN and
 * infinities included, and one of +inf in the sigmoid form (a = 1) keeps it
 * whatever x holds. Behind any other x, gate or state that is not finite h is
 * not finite either, infinite or NaN, up to the next gate of -inf. state_out (fp32
 * [sequences, H, d], NULL: not written) receives the last h in fp32 and may be
 * state_in itself. x, gate and h are [B, H, N, d].
 *
 * Packed sequences: with cu_seqlens (DEVICE int32 [sequences + 1],
 * non-decreasing) B must be 1 and sequence s is tokens cu_seqlens[s] up to
 * cu_seqlens[s + 1] of the one row; max_len bounds the length of a sequence.
 * A sequence may be empty (its state passes through). Tokens outside every
 * sequence, or beyond max_len of one, are neither read nor written. Offsets
 * outside [0, N] are clamped into it. Without cu_seqlens (NULL) `sequences`
 * must be B and max_len N. At most 2^20 sequences, d <= 2^20 and token strides
 * (stride_n) below 2^24 elements, else RET_ERR_UNSUPPORTED, as beyond 2^32
 * threads of a launch (2^26 pieces of 64 channels of a token, say).
 *
 * Gates above 0 in the log form are taken where the products of a channel's
 * decays over up to 256 tokens stay within fp32's range: beyond it h may be inf
 * or NaN where the formula's is finite.
 *
 * workspace: retention_gated_recurrence_workspace_bytes(...) bytes (packed:
 * whether there are cu_seqlens; the same for the backward), 8-byte aligned; its
 * contents on entry do not matter. Calls that may overlap in time need one
 * each: parts of a long sequence wait there for one another. Such a wait ends
 * after a million looks (about a second) whatever happens; the results behind
 * it are then NaN. The first four bytes of the workspace (where the call needs
 * one) say afterwards which it was: all ones where every wait was met, 0 where
 * one was given up, which takes a workspace that something else wrote to
 * during the call, or a GPU that stood still.
 */
size_t retention_gated_recurrence_workspace_bytes(int sequences, int H, int N, int max_len, int packed, int d,
                                                  int dtype);

int retention_gated_recurrence(const retention_view_t* x, const retention_view_t* gate, const retention_view_t* h,
                               int B, int H, int N, int d, int form, int dtype, const float* state_in,
                               float* state_out, const int* cu_seqlens, int sequences, int max_len,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of the recurrence. Given grad_h = dL/dh and grad_state_out =
 * dL/dstate_out (fp32, NULL: 0), with u_t the whole gradient of h_t,
 *   u_t = grad_h_t + a_{t+1} u_{t+1},   u_{last} = grad_h_{last} + grad_state_out
 *   RET_GATE_SIGMOID: grad_x = (1 - a) u, grad_gate = a (1 - a) (h_{t-1} - x_t) u
 *   RET_GATE_LOG:     grad_x = u,         grad_gate = a h_{t-1} u
 *   grad_state_in = a_0 u_0 (fp32; NULL: not written; may be grad_state_out)
 * At a gate of -inf grad_gate and what goes on to the tokens before are 0, at
 * one of +inf in the sigmoid form grad_x and grad_gate, whatever x, h and u hold.
 * h is the forward call's output and state_in its starting state (NULL:
 * zeros); h_{t-1} is read from them, so a bf16 h brings its rounding into
 * grad_gate (RETENTION_H_F32 keeps it out). x may
 * be NULL in the log form, which does not read it. Sequences, cu_seqlens,
 * max_len and the workspace are those of the forward call.
 */
int retention_gated_recurrence_backward(const retention_view_t* grad_h, const retention_view_t* x,
                                        const retention_view_t* gate, const retention_view_t* h,
                                        const retention_view_t* grad_x, const retention_view_t* grad_gate, int B,
                                        int H, int N, int d, int form, int dtype, const float* state_in,
                                        const float* grad_state_out, float* grad_state_in, const int* cu_seqlens,
                                        int sequences, int max_len, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * One token of the recurrence for B rows: h_b = a_b s + (1 - a_b) x_b (or
 * + x_b in the log form), s <- h_b, with s the row's state. Gates of -inf and
 * +inf as over sequences: a slot of any contents is reset by -inf. x, gate and h are
 * [B, H, 1, d]; states is fp32 [nstates, H, d], contiguous. Row b's state is
 * states[b] (nstates >= B) or, with slots (DEVICE int32 [B]), states[slots[b]].
 * A row whose slot is outside [0, nstates) is idle: its h is not written. Rows
 * that name the same slot take effect one after another in row order.
 */
int retention_gated_recurrence_step(const retention_view_t* x, const retention_view_t* gate,
                                    const retention_view_t* h, int B, int H, int d, int form, int dtype,
                                    float* states, int nstates, const int* slots, void* stream);

/* A norm over the d values of a row: layer form ((v - mean) / sqrt(var + eps),
 * biased variance) or, with rms != 0, v / sqrt(mean(v^2) + eps). weight and
 * bias are device fp32 and may each be NULL (1 and 0). */
typedef struct retention_norm_t {
  float eps; /* >= 0 and finite */
  int rms;
  const float* weight;
  const float* bias;
} retention_norm_t;

/*
 * Norm and swish gate after the mixer, per head and token:
 *   y = (norm(o) * weight + bias) * g / (1 + e^-g)
 * o, gate (NULL: no gate) and y are [B, H, N, d]; weight and bias [H * d]. The
 * layer form is what retention_chunkwise applies as its epilogue; as an
 * operator of its own it serves training, where the backward needs o before
 * the norm. d <= RETENTION_MAX_DV, H <= RETENTION_MAX_HEADS.
 */
int retention_gated_norm(const retention_view_t* o, const retention_view_t* gate, const retention_view_t* y, int B,
                         int H, int N, int d, int dtype, const retention_norm_t* norm, void* stream);

/*
 * Gradients of retention_gated_norm for grad_y = dL/dy: grad_o, grad_gate
 * (required with a gate, NULL without), and grad_weight, grad_bias (fp32
 * [H * d], each NULL: not wanted). The statistics are formed again from o. The
 * workspace holds partial sums of the parameter gradients (0 bytes when
 * neither is wanted); its contents on entry do not matter.
 */
size_t retention_gated_norm_backward_workspace_bytes(int B, int H, int N, int d, int dtype, int with_params);

int retention_gated_norm_backward(const retention_view_t* grad_y, const retention_view_t* o,
                                  const retention_view_t* gate, const retention_view_t* grad_o,
                                  const retention_view_t* grad_gate, int B, int H, int N, int d, int dtype,
                                  const retention_norm_t* norm, float* grad_weight, float* grad_bias,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Residual and norm before the next block:
 *   r = alpha * residual + scale * x        y = norm(r) * weight + bias
 * over rows of D <= RETENTION_MAX_MODEL_DIM values. x and y are [B, 1, N, D]
 * of type dtype; residual and r have type stream_dtype, dtype or RET_F32.
 * scale (device fp32 [D], NULL: 1) weighs the branch per channel, alpha
 * (finite) the residual. y is formed from r before its rounding. r may be the
 * residual itself (the same data and strides): the stream is then updated in
 * place.
 */
int retention_residual_norm(const retention_view_t* x, const retention_view_t* residual, const retention_view_t* y,
                            const retention_view_t* r, int B, int N, int D, int dtype, int stream_dtype,
                            const retention_norm_t* norm, const float* scale, float alpha, void* stream);

/*
 * Gradients of retention_residual_norm for grad_y = dL/dy and grad_r = dL/dr
 * (NULL: 0). With t = grad_r + (the norm's gradient for grad_y * weight):
 *   grad_residual = alpha * t (stream_dtype), grad_x = scale * t (dtype),
 *   grad_scale = sum over rows of x * t, grad_weight = sum of grad_y * norm(r),
 *   grad_bias = sum of grad_y   (fp32 [D], each NULL: not wanted)
 * The row that was normed is read from r, the forward call's output, with the
 * rounding it has in the stream's type; with residual (and x) given it is
 * formed again from them instead, and r is not read and may be NULL: with a
 * bf16 stream grad_weight then carries fp32 accuracy. grad_x may be NULL (not
 * wanted, or equal to grad_residual); x is read for grad_scale or with
 * residual only and may be NULL otherwise.
 */
size_t retention_residual_norm_backward_workspace_bytes(int B, int N, int D, int dtype, int with_params);

int retention_residual_norm_backward(const retention_view_t* grad_y, const retention_view_t* grad_r,
                                     const retention_view_t* r, const retention_view_t* x,
                                     const retention_view_t* residual, const retention_view_t* grad_x,
                                     const retention_view_t* grad_residual, int B, int N, int D, int dtype,
                                     int stream_dtype, const retention_norm_t* norm, const float* scale, float alpha,
                                     float* grad_scale, float* grad_weight, float* grad_bias, void* workspace,
                                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RETENTION_BLOCK_H */

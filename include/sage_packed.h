/*
 * sage_packed.h -- C ABI of libsage's 16-bit operators on packed sequences: QK-norm with rotary
 * positions in one pass, and softmax attention over sequences of different lengths laid end to
 * end, with grouped heads, forward and backward.
 *
 * The quantized paths (sage.h, sage_nvfp4.h) work on [B, H, N, d] tensors with N a multiple of
 * 128 and as many key as query heads.  These operators serve the layers and batches around
 * them: layers kept in 16 bits, packed rows of documents or prompts, grouped-query heads, and
 * the rotation of q and k by their positions, which comes between the norm and the attention.
 *
 * Conventions are those of sage.h (device pointers owned by the caller, work asynchronous on
 * `stream`, argument errors returned before any launch, no allocation, no trap, bounded waits),
 * with these additions:
 *   Device     Calls launch on the calling thread's current device, which must be the one
 *              that holds the pointers (and the stream).
 *   Rows       A tensor of vectors is described by sage_rows: the vector of (batch entry b,
 *              token t, head h) has its d channels at ptr + b * batch_stride + t *
 *              token_stride + h * head_stride (elements).  Pointers are 16-byte aligned and
 *              strides multiples of 8 elements, not negative, so q, k and v may be slices of
 *              one projection's output, and [T, H, d] as well as [B, H, N, d] tensors fit.
 *              Outputs must not overlap each other or any input.
 *   Capture    Every call can be captured into a CUDA graph.  Calls that share a workspace
 *              (two captured graphs too) must be ordered by the caller.
 */
#ifndef SAGE_PACKED_H_
#define SAGE_PACKED_H_

#include <stddef.h>
#include <stdint.h>

#include "sage.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  void* ptr;
  int64_t batch_stride, token_stride, head_stride; /* elements */
} sage_rows;

/* ---- QK-norm and rotary positions --------------------------------------------------------- */

/* The vectors of q and k: B batch entries (1 for packed tokens) of N tokens, Hq and Hkv heads.
 * y = R(pos) (x / sqrt(mean_c x_c^2 + eps) * gain): with norm = 0 the normalization and the
 * gains are left out.  R turns pairs of the first rotary_dim channels; pair i is channels
 * (i, i + rotary_dim/2), or (2i, 2i + 1) when interleaved; its angle is pos_a * inv_freq[i]
 * radians, where a is the position axis whose section holds i: the n_axes sections (pairs per
 * axis, none empty, in order) add up to rotary_dim/2.  Turns are 64-bit fixed-point fractions,
 * so full ones drop out exactly, but inv_freq / (2 pi) is rounded to 2^-64 turns (relatively, where
 * it is above 1): the angle is off by up to 2 pi |pos| 2^-64, which passes the kernel's own 2^-20
 * from |pos| = 2^41 on. */
typedef struct {
  int B, N, Hq, Hkv, d;
  int dtype;               /* sage_dtype of x, y and their gradients                      */
  int norm;                /* 1: RMSNorm (and gains), 0: rotation only                    */
  float eps;
  int rotary_dim;          /* multiple of 16, 0 .. d                                      */
  int interleaved;
  int n_axes;              /* 1 .. 4                                                      */
  int sections[4];
  const double* inv_freq;  /* HOST pointer: rotary_dim/2 finite frequencies (read during
                              the call)                                                    */
  int pos_bits;            /* 32 or 64: signed integers                                   */
  int64_t pos_axis_stride, pos_batch_stride; /* elements; token stride 1; a batch stride of
                              0 gives every batch entry the same positions                 */
} sage_rope_params;

/* q_out, k_out: rotated q and k.  gain_q, gain_k: float32 [d], 16-byte
 * aligned (NULL: ones); pos: device.
 * Reads each row once and writes it once; float32 arithmetic, rounded once. */
int sage_qk_norm_rope_fwd(const sage_rope_params* p, const sage_rows* q, const sage_rows* k,
                          const float* gain_q, const float* gain_k, const void* pos,
                          const sage_rows* q_out, const sage_rows* k_out, void* stream);

/* Gradients of sage_qk_norm_rope_fwd for the raw q, k and the gains, given those of its outputs:
 *   g = R^T dy;  dgain_c = sum over tokens and heads of g_c xhat_c;  gx = g gain;
 *   dx = inv (gx - xhat mean_c(gx xhat)).
 * dgain_q, dgain_k (float32 [d], both or none; only with norm): sums in a fixed order, so the
 * result is the same from call to call.  The workspace (16-byte aligned,
 * sage_qk_norm_rope_workspace_bytes) is needed only with dgain. */
size_t sage_qk_norm_rope_workspace_bytes(const sage_rope_params* p);
int sage_qk_norm_rope_bwd(const sage_rope_params* p, const sage_rows* q, const sage_rows* k,
                          const float* gain_q, const float* gain_k, const void* pos,
                          const sage_rows* dq_out, const sage_rows* dk_out, const sage_rows* dq,
                          const sage_rows* dk, float* dgain_q, float* dgain_k, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ---- packed attention --------------------------------------------------------------------- */

/* S sequences of lengths[0 .. S-1] >= 0 tokens laid end to end in T >= sum(lengths) rows.  The
 * plan lists their tiles of 128 tokens, largest work first, for the kernels' CTAs.  Tiles are
 * cut from a sequence's end, so that only its first tile can be ragged.  Built on the host:
 * sage_packed_plan_bytes gives the size (0: no sequence, a negative length, or 2^31 - 128 tokens or more in all),
 * sage_packed_plan_fill writes it to host memory, and the caller copies those bytes to the
 * device (16-byte aligned) and gives that copy's address, with what fill returned in `info`, to
 * every call on batches of these lengths.  The plan is read-only. */
typedef struct {
  int sequences, tiles, pairs, longest; /* longest: tokens of the longest sequence  */
  int64_t tokens;                       /* sum of the lengths */
  int64_t causal_steps, full_steps;     /* (query tile, key tile) pairs of one head */
} sage_packed_info;

size_t sage_packed_plan_bytes(const int* lengths, int sequences);
int sage_packed_plan_fill(const int* lengths, int sequences, void* host_plan, size_t bytes,
                          sage_packed_info* info);

typedef struct {
  int64_t T;          /* rows of every tensor, >= info.tokens; below 2^31 */
  int Hq, Hkv, d;     /* Hq a multiple of Hkv; query head h reads key head h / (Hq / Hkv) */
  int dtype, causal;  /* causal: token i of a sequence sees its tokens 0 .. i */
  float softmax_scale; /* <= 0: 1/sqrt(d) */
} sage_packed_params;

/* Forward: o = softmax(softmax_scale q k^T) v within each sequence; lse [Hq][T] float32, the
 * natural log-sum-exp of the scaled scores.  Products of 16-bit values summed in float32; P is
 * rounded to dtype for the product with v.  Rows behind the last sequence are neither read
 * nor written.  Sequences never affect each other, whatever their values.  A row that
 * sees a score of NaN or +inf is NaN in o and lse; a score of -inf weighs nothing, and a row with
 * no other has o = NaN, lse = -inf.  A value that is not finite may also reach rows of its own
 * sequence that do not see it, as 0 * inf.  The workspace (16-byte aligned) is needed where
 * sage_packed_attn_fwd_workspace_bytes is not 0: few heads and long sequences, whose walks over
 * the keys are cut into parts and joined. */
size_t sage_packed_attn_fwd_workspace_bytes(const sage_packed_params* p,
                                            const sage_packed_info* info);
int sage_packed_attn_fwd(const sage_packed_params* p, const sage_packed_info* info,
                         const void* plan, const sage_rows* q, const sage_rows* k,
                         const sage_rows* v, const sage_rows* o, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Backward from the forward's o and lse: dq, dk, dv (workspace 16-byte aligned).  A query head's score gradient is
 * rounded to dtype for its products; each key head's gradients sum over its query heads in
 * float32, in a fixed order: results are the same from call to call. */
size_t sage_packed_attn_bwd_workspace_bytes(const sage_packed_params* p,
                                            const sage_packed_info* info);
int sage_packed_attn_bwd(const sage_packed_params* p, const sage_packed_info* info,
                         const void* plan, const sage_rows* q, const sage_rows* k,
                         const sage_rows* v, const sage_rows* o, const float* lse,
                         const sage_rows* dout, const sage_rows* dq, const sage_rows* dk,
                         const sage_rows* dv, void* workspace, size_t workspace_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SAGE_PACKED_H_ */

/*
 * gdn_glr.h -- gated linear recurrence with a vector state (sm_100a).
 *
 * The companion of the Gated DeltaNet layer whose state is a vector: every
 * channel c of every sequence runs
 *
 *     h_t = a_t h_{t-1} + b_t,   a_t = exp(g_t),
 *     b_t = x_t                 (GDN_GLR_INPUT_PLAIN)
 *     b_t = (1 - a_t) x_t       (GDN_GLR_INPUT_COMPLEMENT)
 *
 * with its own gate per token and channel.  It keeps the promise of section
 * "Solving the linear-attention headache" of "NovaSky's IsoExec Fixes the
 * Hidden Math Bug Corrupting AI Training Runs" for this recurrence too:
 * prefill, trainer forward and decode share one rounding schedule, so their
 * outputs are bitwise identical and independent of the batch.  (The pages
 * treat the matrix state only.)
 *
 * The schedule.  Chunks of GDN_GLR_CHUNK tokens start at each sequence's
 * first token.  Inside a chunk entered with state H (all fp32, round to
 * nearest, A = 1 and B = 0 at the chunk's start):
 *     A <- a_t A,   B <- fma(a_t, B, b_t),   h_t = fma(A, H, B)
 * and the next chunk's H is the last h_t.  A and B do not depend on H, so
 * the chunks of a sequence are evaluated side by side.
 *
 * Conventions are those of gdn_cpr.h (device pointers of the current device,
 * caller-owned memory, argument errors before any launch, device error word,
 * no float atomics) with these differences: x, g, h and their gradients
 * [tokens, D] may have a row stride (ld*, in elements, >= D); they and the
 * contiguous fp32 arrays [rows, D] need only the alignment of their elements
 * (16 bytes for a decode state).  Rows that start on 16 bytes are the fast ones.
 * g may be -inf; it must not be NaN or +inf.  An a below 2^-126 counts as 0.
 * Gates may grow (g > 0) as long as A stays in fp32's range: the sum of g over
 * the first tokens of a chunk, up to any of them, stays below 88 (16 gates of
 * 5.5).  Beyond that A is infinite, and h is NaN where the state that entered
 * the chunk is 0, or after a reset in the same chunk.
 * D is any size from 1 to 2^24, total_tokens up to 2^31 - 4097, strides up to
 * 2^27 elements, n_seqs ceil(D / 32) up to 2^28 - 1.
 */
#ifndef GDN_GLR_H
#define GDN_GLR_H

#include <stddef.h>
#include <stdint.h>

#include "gdn_cpr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_GLR_CHUNK 16
#define GDN_GLR_TILE 128 /* tokens between two rows of the carry */

typedef enum { GDN_GLR_INPUT_PLAIN = 0, GDN_GLR_INPUT_COMPLEMENT = 1 } gdn_glr_input;

/*
 * Decode state of n_slots sequences (caller-owned device arrays):
 *   h      [n_slots, D] fp32  state that entered the current chunk
 *   a, b   [n_slots, D] fp32  A and B of the chunk's tokens so far (their
 *                             values are not used when pos == 0)
 *   pos    [n_slots] int32    tokens already in the chunk, 0 .. 15
 *   error  [1] int32          device error word (GDN_DEVERR_* bits)
 * The state itself is h when pos == 0, else fma(a, h, b).  A sequence that
 * starts from h0 has h = h0 and pos = 0.
 */
typedef struct {
  float* h;
  float* a;
  float* b;
  int32_t* pos;
  int32_t* error;
  int n_slots;
} gdn_glr_state;

/* Rows of the carry gdn_glr_forward writes and gdn_glr_backward reads; 0 for
 * arguments gdn_glr_forward would reject. */
int64_t gdn_glr_carry_rows(int n_seqs, int64_t total_tokens);

/*
 * gdn_glr_forward -- the recurrence over packed variable-length sequences.
 *
 * x           [total_tokens, D] in_dtype, row stride ldx
 * g           [total_tokens, D] g_dtype (GDN_BF16 or GDN_F32), row stride ldg
 * cu_seqlens  [n_seqs + 1] int32 on the device, as for gdn_cpr_forward
 * h0          [n_seqs, D] fp32 initial states, or NULL for zeros
 * h           [total_tokens, D] out_dtype, row stride ldh: h_t of every token
 * s_final     [n_seqs, D] fp32 or NULL: the state after each sequence's last
 *             token (h0 for an empty one)
 * state       NULL, or the decode state that receives every sequence's final
 *             (h, a, b, pos), from which gdn_glr_decode_step continues bit
 *             for bit: sequence n goes to slot slot_idx[n] (slot n when
 *             slot_idx is NULL).  A slot outside [0, n_slots), or one that an
 *             earlier sequence of the call names too, is not written and sets
 *             GDN_DEVERR_POS in state->error.
 * carry       [gdn_glr_carry_rows, D] fp32 or NULL: the states at the tile
 *             starts, which gdn_glr_backward needs
 * error_word  optional device int32 (4-byte aligned), cleared by the call;
 *             invalid cu_seqlens set GDN_DEVERR_CU_SEQLENS there.  A sequence
 *             that ends before it starts, or leaves the batch, is not
 *             written; what the call's outputs hold for the others, which
 *             may overlap then, is not specified.  Nothing but the outputs is
 *             written.
 * A forward over a prefix whose length is a multiple of GDN_GLR_CHUNK,
 * followed by one over the rest with h0 = s_final, gives the bits of one
 * forward over the whole.  n_seqs may be 0 and sequences may be empty.
 * Outputs must not overlap the inputs.
 */
int gdn_glr_forward(const void* x, int64_t ldx, int in_dtype, const void* g, int64_t ldg,
                    int g_dtype, const int32_t* cu_seqlens, int n_seqs, int64_t total_tokens,
                    int D, int input_mode, const float* h0, void* h, int64_t ldh, int out_dtype,
                    float* s_final, const gdn_glr_state* state, const int32_t* slot_idx,
                    float* carry, int32_t* error_word, void* stream);

/*
 * gdn_glr_backward -- reverse mode of gdn_glr_forward for a loss
 * L(h, s_final):
 *     lam_t = dL/dh_t + mu_{t+1},   mu_t = a_t lam_t,
 *     (the last token's mu_{t+1} is dL/ds_final)
 *     PLAIN:       dx_t = lam_t,             dg_t = mu_t h_{t-1}
 *     COMPLEMENT:  dx_t = (1 - a_t) lam_t,   dg_t = mu_t (h_{t-1} - x_t)
 *     dh0 = mu of the first token (dL/ds_final for an empty sequence)
 * h_{t-1} is recomputed in fp32 from the carry, bitwise the forward's.
 *
 * x, g, cu_seqlens, n_seqs, total_tokens, D, input_mode: as for the forward
 * carry     [gdn_glr_carry_rows, D] fp32 as the forward of the same x, g,
 *           cu_seqlens and h0 wrote it (the library cannot check that)
 * d_h       [total_tokens, D] dh_dtype, row stride lddh: dL/dh
 * ds_final  [n_seqs, D] fp32 dL/ds_final, or NULL for zeros
 * d_x       [total_tokens, D] in_dtype, row stride lddx
 * d_g       [total_tokens, D] g_dtype, row stride lddg
 * d_h0      [n_seqs, D] fp32 or NULL
 * error_word as for the forward.
 * Every sum has a fixed order: repeated calls, and any batch composition,
 * give identical bits.  Outputs must not overlap the inputs.
 */
int gdn_glr_backward(const void* x, int64_t ldx, int in_dtype, const void* g, int64_t ldg,
                     int g_dtype, const int32_t* cu_seqlens, int n_seqs, int64_t total_tokens,
                     int D, int input_mode, const float* carry, const void* d_h, int64_t lddh,
                     int dh_dtype, const float* ds_final, void* d_x, int64_t lddx, void* d_g,
                     int64_t lddg, float* d_h0, int32_t* error_word, void* stream);

/*
 * gdn_glr_decode_step -- one token for each of B rows: row b advances slot
 * slot_idx[b] (slot b when slot_idx is NULL) and writes h[b], bitwise what
 * gdn_glr_forward over the whole sequence gives for that token.  When the
 * token fills its chunk, state.h receives h, a becomes 1, b becomes 0 and
 * pos returns to 0.
 * x [B, D] in_dtype, g [B, D] g_dtype, h [B, D] out_dtype, row strides as
 * above.  A row whose slot is outside [0, n_slots), whose slot an earlier
 * row of the call names too, or whose pos is outside [0, GDN_GLR_CHUNK)
 * writes nothing and sets GDN_DEVERR_POS in state.error.
 * The launch depends only on the arguments' sizes, so the call can be
 * captured in a CUDA graph.
 */
int gdn_glr_decode_step(const void* x, int64_t ldx, int in_dtype, const void* g, int64_t ldg,
                        int g_dtype, const int32_t* slot_idx, int B, int D, int input_mode,
                        gdn_glr_state state, void* h, int64_t ldh, int out_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_GLR_H */

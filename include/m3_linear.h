/*
 * m3_linear.h -- C ABI of linear attention with a decay for each head (AMD
 * MI355X / gfx950): the prompt pass over packed sequences, its gradients and
 * the single-token step.
 *
 * With H = max(q_heads, k_heads, v_heads) heads, each of the three counts
 * dividing H (head h reads row h / (H / q_heads) of q, and k and v likewise),
 * g_h = exp(log_decay[h]) and a key_dim x value_dim state S per sequence and
 * head:
 *     S_t = g S_{t-1} + k_t v_t^T,        o_t = scale * q_t^T S_t.
 * The prompt pass works in chunks of tokens; for row r of a chunk that starts
 * with state S,
 *     o_r = scale (sum_{s<=r} g^{r-s} (q_r . k_s) v_s + g^{r+1} q_r^T S),
 * and the state moves on by the chunk's weighted sum of k v^T.
 *
 * Rows and strides.  q, k, v and o are rows [token][head][channel] with the
 * channels of one row contiguous; an m3_rows_t names the strides of the other
 * two axes in elements, so views of one projection's rows are taken as they
 * are.  Rows must be 16-byte aligned: the base pointer, and both strides
 * multiples of 8 elements.  The tokens' stride is at least the row's channels
 * and below 2^24 (of no account with one token), the heads' from 0 to below
 * 2^40.
 *
 * Sequences.  cu_seqlens (device, int32, batch + 1 entries, ascending from 0
 * to at most `tokens`) gives sequence b the tokens cu_seqlens[b] up to
 * cu_seqlens[b + 1]; a sequence may have no token.  NULL: `batch` sequences
 * of tokens / batch tokens each.  Tokens outside every sequence are not read,
 * and their rows of o are left as they were.  Entries are clamped to
 * [0, tokens]; entries that do not ascend give unspecified values.
 *
 * States are [n][H][key_dim][value_dim], contiguous, 16-byte aligned, in
 * state_dtype (arithmetic is fp32; bf16 is rounded to nearest even once per
 * call).  slots (device, int32, batch entries, or NULL: sequence b has state
 * b) names each sequence's state among the nstates of the pool (where no state
 * is read or written, any count that the slots stay below).  A sequence whose
 * slot is negative or not below nstates is padding: nothing of it is
 * read, and its rows of o are left as they were.  When two sequences of one
 * call name the same slot, the first has it; the rows of o of the later ones
 * are filled with NaN.
 *
 * log_decay is a constant of the layer, at most 0 (not checked; -inf forgets
 * everything before the token itself).  The weights of a chunk are taken in
 * fp32 from it, and no gradient is formed for it.  A non-finite value of one
 * token reaches, within its sequence and head, the outputs of its own chunk
 * (at most 64 tokens; counted from the end of the sequence for the gradients
 * of k and v) and of everything behind it, and no other sequence.  It may
 * arrive as NaN where it was an infinity; an infinite entry of a state stays
 * one, or becomes NaN where the decay of a chunk is zero in fp32.
 *
 * Ownership, streams, threads and errors are those of m3_ssm.h: the caller
 * owns every buffer and the workspace, calls only enqueue kernels, nothing is
 * allocated or synchronised, a workspace needs no initialisation and serves
 * one call at a time.  Outputs must not overlap inputs or each other, except
 * that final_state may be init; M3_ERR_INVALID_ARGUMENT where one starts at
 * another's address.
 */
#ifndef M3_LINEAR_H
#define M3_LINEAR_H

#include "m3_ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows [token][head][channel]: strides in elements, channels contiguous. */
typedef struct {
    void *data;
    int64_t token_stride;
    int64_t head_stride;
} m3_rows_t;

/* Supported: key_dim and value_dim multiples of 8 from 8 to 128; any head
 * counts that divide the largest; batch >= 1; tokens >= 0 (decode: ignored,
 * there is one token per sequence).  M3_ERR_INVALID_ARGUMENT for counts that
 * do not divide, M3_ERR_UNSUPPORTED for other sizes, for H times key_dim or
 * value_dim from 2^24 on, and for more sequences,
 * tokens and heads than one launch has threads for: (batch + 8 + tokens / 1024)
 * H up to 2795690, for a decode step (batch + 8) H up to 8388095. */
typedef struct {
    int64_t batch;      /* sequences                                              */
    int64_t tokens;     /* rows of q, k, v and o                                  */
    int64_t max_seqlen; /* longest sequence, to plan by (any value is right; 0 = tokens) */
    int32_t q_heads, k_heads, v_heads;
    int32_t key_dim, value_dim;
    int32_t io_dtype;    /* m3_dtype_t of q, k, v, o and their gradients           */
    int32_t state_dtype; /* m3_dtype_t of the states                               */
    float scale;         /* factor of o                                            */
} m3_linear_shape_t;

/* Bytes of device workspace m3_linear_prefill needs (0: invalid or unsupported
 * shape).  Where the sequences and heads alone do not fill the chip, sequences
 * are cut into segments, and the workspace holds one fp32 state per segment
 * and head; otherwise it is 256 bytes, unused.  With L tokens a segment
 * (m3_linear_plan) that is at most the smaller of tokens / L + batch and
 * 2 tokens / L states of every head.  Without max_seqlen one sequence may be
 * all tokens, so that batches are cut that need not be: 256 sequences of 2048
 * tokens of 64 x 128 x 128 then take 3.2 GB, with it 256 bytes. */
size_t m3_linear_prefill_workspace_bytes(const m3_linear_shape_t *shape);

/* Tokens per segment of the prompt pass (0: sequences are not cut), and of the
 * gradients' passes.  Either pointer may be NULL. */
m3_status_t m3_linear_plan(const m3_linear_shape_t *shape, int64_t *prefill_segment, int64_t *backward_segment);

/*
 * Prompt pass.
 *   init         NULL: every sequence starts from zero; else the states to start from.
 *   final_state  NULL: not written; else receives the state behind each sequence's
 *                last token (of an empty sequence: its initial state); may be init.
 */
m3_status_t m3_linear_prefill(const m3_linear_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                              const m3_rows_t *v, const float *log_decay, const int32_t *cu_seqlens,
                              const int32_t *slots, int64_t nstates, const void *init, void *final_state,
                              const m3_rows_t *o, void *workspace, size_t workspace_bytes,
                              hipStream_t stream);

/* One token of every sequence (row b of q, k, v, o: sequence b), updating the
 * states in place.  tokens and max_seqlen of the shape are ignored. */
m3_status_t m3_linear_decode_step(const m3_linear_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                                  const m3_rows_t *v, const float *log_decay, const int32_t *slots,
                                  int64_t nstates, void *state, const m3_rows_t *o, hipStream_t stream);

/* Bytes of device workspace m3_linear_prefill_backward needs: segment states
 * for the two directions and, for rows shared by several heads, the heads'
 * parts of their gradients in fp32. */
size_t m3_linear_prefill_backward_workspace_bytes(const m3_linear_shape_t *shape);

/*
 * Gradients of L = sum(go * o) + <gfinal, final state> for the prompt pass.
 *   init     the initial states of the pass ([batch] states, state_dtype) or NULL.
 *   go       rows [token][H][value_dim].
 *   gfinal   [batch][H][key_dim][value_dim] fp32, or NULL: zero.
 *   gq,gk,gv rows like q, k, v, each rounded once to io_dtype; the gradients of
 *            a row that several heads share are summed in fp32.  Rows of tokens
 *            outside every sequence are set to zero.
 *   ginit    gradient of init, like gfinal, or NULL: not written.
 *            Where it is asked for, bf16 gradients of rows may be rounded
 *            otherwise in their last bit.
 */
m3_status_t m3_linear_prefill_backward(const m3_linear_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                                       const m3_rows_t *v, const float *log_decay, const int32_t *cu_seqlens,
                                       const void *init, const m3_rows_t *go, const float *gfinal,
                                       const m3_rows_t *gq, const m3_rows_t *gk, const m3_rows_t *gv,
                                       float *ginit, void *workspace, size_t workspace_bytes,
                                       hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* M3_LINEAR_H */

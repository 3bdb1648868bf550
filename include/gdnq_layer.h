/*
 * gdnq_layer.h -- C ABI of libgdnq, part 4: the operators that stand around the recurrence in a
 * layer, forward and backward, for NVIDIA B200 (sm_100a):
 *   gdn_short_conv   the causal depthwise convolution in front of q, k, v (or of a gated scan)
 *   gdn_gated_scan   the gated linear recurrence with a vector state per head
 *   gdn_group_norm   the norm over each head's channels, with an activation or a gate, behind it
 *
 * Conventions are those of gdnq.h (device pointers, caller-owned buffers, asynchronous work on
 * `stream`, argument checks before anything is enqueued, an empty batch a valid call), and:
 *   - A token array is described by a gdn_tokens and holds elements (b, l, h, d): sequence b < B,
 *     token l < L, head h < H, channel d < D, at ptr[b sb + l sl + h sh + d]. Dense [B][L][H][D]
 *     has (L H D, H D, D), what gdn_prefill takes and leaves, [B][H][L][D], has (H L D, D, L D), a
 *     slice of a projection's rows has the row's length as sl. Strides are in elements and >= 0;
 *     an input may repeat elements (stride 0), an output may not.
 *   - An output may not overlap an input or another output, except where a call says so. That is
 *     refused (GDN_ERR_INVALID_ARG) where one of the two has no gaps between its elements or both
 *     have the same strides; two arrays with gaps and different strides are the caller's to keep apart.
 *   - lens (device int32 [B], or NULL: every sequence has L tokens) gives the tokens of each
 *     sequence of a padded batch, each value taken into [0, L]. What stands in the arrays behind a
 *     sequence's end is neither read nor written.
 *   - Activations (GDN_DTYPE_BF16 or GDN_DTYPE_F32) are rounded once, to nearest even, when they
 *     are stored; parameters, their gradients, log-gates and scan states are fp32, and all
 *     arithmetic is fp32. Results do not depend on the order in which CTAs run.
 *   - Sizes: L <= 2^30, H D <= 2^30, B H < 2^31, B H D <= 2^36; offsets inside arrays are 64-bit,
 *     tokens at most 2^27 elements apart (GDN_ERR_UNSUPPORTED beyond).
 *   - Errors: GDN_ERR_INVALID_ARG for a null or misaligned pointer, a bad size, stride or enum
 *     value, or a workspace too small; GDN_ERR_UNSUPPORTED for a size that is not built;
 *     GDN_ERR_CUDA for a failed launch.
 */
#ifndef GDNQ_LAYER_H
#define GDNQ_LAYER_H

#include "gdnq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    void* ptr;          /* element (0, 0, 0, 0); aligned to its element */
    int64_t sb, sl, sh; /* elements from one sequence, token, head to the next */
} gdn_tokens;

typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1, GDN_ACT_SIGMOID = 2 } gdn_activation;

/* ---- gated scan --------------------------------------------------------------------------- */

/* The factor s(g) of the scan's input. */
typedef enum {
    GDN_SCALE_NONE = 0,       /* 1 */
    GDN_SCALE_COMPLEMENT = 1, /* 1 - e^g: the state is a running average */
    GDN_SCALE_SQRT = 2        /* sqrt(1 - e^{2g}), g <= 0: the state keeps the input's variance */
} gdn_input_scale;

typedef struct {
    int32_t B, H, D;   /* sequences, heads, channels of a head (D >= 1) */
    int32_t scale;     /* gdn_input_scale */
    int32_t act_dtype; /* gdn_dtype of x, o and their gradients */
} gdn_scan_config;

/* Tokens between the states that gdn_gated_scan keeps for its backward pass. */
#define GDN_SCAN_CHUNK 64

/* Shorter sequences are never split: gdn_gated_scan and its backward need no workspace for them. */
#define GDN_SCAN_SPLIT 4096

/*
 * L tokens of the gated linear recurrence of every (sequence, head, channel), whose state is one
 * number (the matrix state of gdnq.h without keys and queries):
 *     h_t = a_t h_{t-1} + s(g_t) x_t,   a_t = e^{g_t},   o_t = h_t.
 * g_t = -inf forgets all before (the first token of a document in a packed row); g_t = 0 with
 * x_t = 0 changes nothing. Runs of tokens are joined by the products of their gates: a gate above 1
 * (g_t > 0, not with GDN_SCALE_SQRT) is taken too, as long as in no stretch of up to 1024 tokens the
 * gates' logs sum to 88 or more. A gate, or a product of successive tokens' gates, below 2^-126 may
 * count as zero.
 *   x     act tokens;  g  fp32 tokens, the log of the gate;  o  act tokens, written.
 *   h0    fp32 [B][H][D], the states before the first token, or NULL: zero.
 *   hT    fp32 [B][H][D], the states after each sequence's last token, or NULL; may be h0.
 *   hist  fp32 [B][ceil(L / GDN_SCAN_CHUNK)][H][D], or NULL: the state before every 64th token,
 *         for gdn_gated_scan_backward. Chunks that begin at or behind a sequence's end are not
 *         written.
 *   workspace  16-byte aligned, at least gdn_gated_scan_workspace_bytes(cfg, L) bytes (may be NULL
 *         where that is 0): few and long sequences are split, and their parts' effects on the
 *         state kept there. Contents are ignored on entry; calls whose work may overlap in time
 *         need workspaces of their own.
 * L = 1 is the decode step.
 */
gdn_status gdn_gated_scan(const gdn_scan_config* cfg, int32_t L, const gdn_tokens* x,
                          const gdn_tokens* g, const gdn_tokens* o, const float* h0, float* hT,
                          float* hist, const int32_t* lens, void* workspace,
                          size_t workspace_bytes, gdn_stream_t stream);

/* Bytes of workspace that gdn_gated_scan and gdn_gated_scan_backward need (0 for most sizes, and for
 * a cfg that they reject). Host-only. */
size_t gdn_gated_scan_workspace_bytes(const gdn_scan_config* cfg, int32_t L);

/*
 * Gradients of gdn_gated_scan, from grad_o (the gradient of o) and grad_hT (that of hT, or NULL:
 * zero). With dh_t the gradient of h_t:
 *     dh_t = grad_o_t + a_{t+1} dh_{t+1}   (grad_o_t + grad_hT_t at a sequence's last token)
 *     grad_x_t = s(g_t) dh_t,   grad_g_t = a_t h_{t-1} dh_t + s'(g_t) x_t dh_t,
 *     grad_h0 = a_1 dh_1   (grad_hT for a sequence of no tokens).
 * s'(0) of GDN_SCALE_SQRT, where the root has no derivative, is taken as 0.
 *   x, g, lens, workspace as in the forward call; hist what that call wrote.
 *   grad_x act tokens, grad_g fp32 tokens, grad_h0 fp32 [B][H][D] or NULL (may be grad_hT): written.
 */
gdn_status gdn_gated_scan_backward(const gdn_scan_config* cfg, int32_t L, const gdn_tokens* x,
                                   const gdn_tokens* g, const float* hist,
                                   const gdn_tokens* grad_o, const float* grad_hT,
                                   const gdn_tokens* grad_x, const gdn_tokens* grad_g,
                                   float* grad_h0, const int32_t* lens, void* workspace,
                                   size_t workspace_bytes, gdn_stream_t stream);

/* ---- group norm --------------------------------------------------------------------------- */

/* Largest D of gdn_group_norm. */
#define GDN_NORM_MAX_D 8192

typedef enum { GDN_WEIGHT_HEAD = 0, GDN_WEIGHT_CHANNEL = 1 } gdn_weight_kind;

typedef struct {
    int32_t B, H, D;    /* sequences, heads (groups), channels of a head, D <= GDN_NORM_MAX_D */
    int32_t center;     /* 1: the mean is taken off (group norm); 0: it is not (RMS norm) */
    int32_t activation; /* gdn_activation */
    int32_t weight;     /* gdn_weight_kind: w and bias [D], shared by the heads, or [H][D] */
    int32_t act_dtype;  /* gdn_dtype of x, z, y and their gradients */
    float eps;          /* > 0 */
} gdn_norm_config;

/*
 * For every token and head, over the head's D channels, with m their mean (0 without center):
 *     n = (x - m) / sqrt(mean((x - m)^2) + eps),   u = n w + bias,
 *     y = act(u) without a gate z,   y = u act(z) with one.
 *   x act tokens, w fp32, bias fp32 or NULL, z act tokens or NULL, y act tokens (written).
 */
gdn_status gdn_group_norm(const gdn_norm_config* cfg, int32_t L, const gdn_tokens* x,
                          const float* w, const float* bias, const gdn_tokens* z,
                          const gdn_tokens* y, const int32_t* lens, gdn_stream_t stream);

/*
 * Gradients of gdn_group_norm from grad_y; the statistics are taken from x again:
 *     du = grad_y act'(u)  (grad_y act(z) with a gate),   grad_z = grad_y u act'(z),
 *     dn = du w,   grad_x = (dn - [center] mean(dn) - n mean(dn n)) / sqrt(mean((x - m)^2) + eps),
 *     grad_w = sum du n,   grad_bias = sum du   over all tokens (and heads for a shared weight).
 *   grad_x and (with z) grad_z act tokens, grad_w like w, grad_bias like bias (NULL exactly when
 *   bias is NULL; grad_z NULL exactly when z is): written.
 *   workspace  16-byte aligned, at least gdn_group_norm_backward_workspace_bytes(cfg, L) bytes:
 *   partial sums of the parameters' gradients. Contents are ignored on entry; calls whose work
 *   may overlap in time need workspaces of their own.
 */
gdn_status gdn_group_norm_backward(const gdn_norm_config* cfg, int32_t L, const gdn_tokens* x,
                                   const float* w, const float* bias, const gdn_tokens* z,
                                   const gdn_tokens* grad_y, const gdn_tokens* grad_x,
                                   const gdn_tokens* grad_z, float* grad_w, float* grad_bias,
                                   const int32_t* lens, void* workspace, size_t workspace_bytes,
                                   gdn_stream_t stream);

/* Bytes of workspace the call above needs (0 for a cfg that it rejects). Host-only. */
size_t gdn_group_norm_backward_workspace_bytes(const gdn_norm_config* cfg, int32_t L);

/* ---- short convolution ---------------------------------------------------------------------- */

/* Largest K of gdn_short_conv. */
#define GDN_CONV_MAX_K 4

typedef struct {
    int32_t B, H, D;    /* sequences, heads, channels of a head (D >= 1) */
    int32_t K;          /* taps, 2 <= K <= GDN_CONV_MAX_K */
    int32_t activation; /* GDN_ACT_NONE or GDN_ACT_SILU */
    int32_t act_dtype;  /* gdn_dtype of x, y, the states and their gradients */
} gdn_conv_config;

/*
 * The causal depthwise convolution of every (head, channel) c over the tokens of its sequence:
 *     p_t = bias[c] + sum_{j < K} w[c][j] x_{t-K+1+j},   y_t = act(p_t),
 * where the K - 1 inputs before the first token come from state_in.
 *   x act tokens, w fp32 [H][D][K], bias fp32 [H][D] or NULL, y act tokens (written).
 *   state_in   act [B][K-1][H][D], oldest first, or NULL: zero.
 *   state_out  act [B][K-1][H][D], or NULL: the last K - 1 inputs of each sequence (those of
 *              state_in among them when it has fewer tokens); may be state_in.
 * L = 1 is the decode step.
 */
gdn_status gdn_short_conv(const gdn_conv_config* cfg, int32_t L, const gdn_tokens* x,
                          const float* w, const float* bias, const void* state_in,
                          const gdn_tokens* y, void* state_out, const int32_t* lens,
                          gdn_stream_t stream);

/*
 * Gradients of gdn_short_conv from grad_y and grad_state_out (or NULL: zero):
 *     dp_t = grad_y_t act'(p_t),   grad_x_s = sum_j w[c][j] dp_{s+K-1-j}, and what grad_state_out
 *     has for token s,   grad_w[c][j] = sum dp_t x_{t-K+1+j},   grad_bias[c] = sum dp_t;
 * grad_state_in is grad_x of the K - 1 inputs before the first token.
 *   x, w, bias, state_in, lens as in the forward call. grad_x act tokens, grad_w fp32 [H][D][K],
 *   grad_bias fp32 [H][D] (NULL exactly when bias is NULL), grad_state_in act [B][K-1][H][D] or
 *   NULL: written.
 *   workspace as for gdn_group_norm_backward.
 */
gdn_status gdn_short_conv_backward(const gdn_conv_config* cfg, int32_t L, const gdn_tokens* x,
                                   const float* w, const float* bias, const void* state_in,
                                   const gdn_tokens* grad_y, const void* grad_state_out,
                                   const gdn_tokens* grad_x, float* grad_w, float* grad_bias,
                                   void* grad_state_in, const int32_t* lens, void* workspace,
                                   size_t workspace_bytes, gdn_stream_t stream);

size_t gdn_short_conv_backward_workspace_bytes(const gdn_conv_config* cfg, int32_t L);

#ifdef __cplusplus
}
#endif

#endif /* GDNQ_LAYER_H */

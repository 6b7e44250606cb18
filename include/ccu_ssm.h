/*
 * ccu_ssm -- the operators around the short causal convolution of a state-space layer, for
 * NVIDIA GB300 (sm_103a): the convolution over packed prompts, the selective scan over
 * packed prompts, the selective state update of one token per row, and products with
 * 4-bit weights; the gated delta rule, the other recurrence behind that convolution, over packed prompts and for one
 * token per row; and the norms around such a layer.
 *
 * The conventions of ccu_conv1d.h hold here too: tensor pointers are device memory owned
 * by the caller; nothing is allocated, copied to the host or synchronized; calls only
 * enqueue kernels on `stream` and can be captured in a CUDA graph (make one call of the
 * same kind on the device before the capture); every argument is checked before any launch
 * and a declined call changes nothing; sizes and strides are elements; the message of a
 * decline is read with ccu_conv1d_last_error().
 *
 * Arguments are passed in one struct per operator. Zero the struct first (memset), then set
 * the members: NULL or 0 is the documented default of everything optional.
 *
 * Packed sequences: the T token rows of a call hold B sequences one after the other;
 * sequence b is the rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 (int32 [B + 1] on the device,
 * ascending from 0; equal neighbours are an empty sequence). Each sequence's offsets are clamped to [0, T] and its end to its
 * begin or more before they are used: offsets that do not ascend reach no memory outside the tensors, but which of their sequences are
 * computed, and what from, is not defined. Output rows outside every sequence are not written.
 *
 * Slots: sequence (or row) i keeps its state in cache slot indices[i], or in slot i when
 * indices is NULL. A slot of -1 marks padding: its outputs are +0 and no state is read or written.
 * A slot below -1 or >= S is treated as padding and, with a status word, reported as
 * CCU_DEVERR_RANGE. A slot may be used by one sequence of a call only (not checked; see
 * ccu_conv1d_check_indices).
 */
#ifndef CCU_SSM_H
#define CCU_SSM_H

#include "ccu_conv1d.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ccu_causal_conv1d_packed -- the causal depthwise convolution over packed prompts, with the
 * convolution state of every sequence read from and left in its cache slot.
 *
 *   out[t, d] = act( sum_{j=0}^{W-1} weight[d, j] * u(t - (W-1) + j) + bias[d] )
 *
 * where u is x inside t's sequence, before its first row the entries of the slot's state
 * (newest last) when has_initial[b] != 0, and zero otherwise. The state after the sequence,
 * the last L entries of its inputs (preceded by the old state, or zeros), goes to
 * the slot: what ccu_conv1d_update continues from. Arithmetic and rounding are those of
 * ccu_causal_conv1d_fwd.
 */
typedef struct ccu_conv1d_packed_args {
  const void *x;             /* BF16 [T, D], row stride ld_x, unit stride along D */
  int64_t ld_x;
  const void *weight;        /* BF16 contiguous [D, W] */
  const void *bias;          /* BF16 [D] or NULL */
  void *conv_state;          /* BF16 [S, D, L] by strides, or NULL: no states */
  int64_t stride_s, stride_d, stride_l;
  const int32_t *cu_seqlens; /* int32 [B + 1] */
  const int32_t *indices;    /* int32 [B] or NULL */
  const int32_t *has_initial; /* int32 [B] or NULL (no sequence has one) */
  void *out;                 /* BF16 [T, D], row stride ld_out; must not overlap x */
  int64_t ld_out;
  int32_t *status_dev;       /* device word for CCU_DEVERR_RANGE, or NULL */
  int64_t T, B, D, S, L, W;  /* T < 2^31; W = 2..4, L >= W - 1 (L ignored without conv_state) */
  int32_t act;               /* ccu_act_t */
  int32_t reserved;          /* 0 */
} ccu_conv1d_packed_args_t;

CCU_API ccu_status_t ccu_causal_conv1d_packed(const ccu_conv1d_packed_args_t *args, ccu_stream_t stream);

/*
 * ccu_selective_scan -- the selective state space scan over packed prompts.
 *
 * Per head h (its group g = h / (H / G)) a matrix state s[P, K] runs over the tokens of a
 * sequence:
 *
 *   d       = softplus(dt[t, h] + dt_bias[h])      (dt + dt_bias when dt_softplus is 0)
 *   s[p, k] = exp(d * A[h]) * s[p, k] + d * x[t, h, p] * B[t, g, k]
 *   y[p]    = sum_k C[t, g, k] * s[p, k] + D[h] * x[t, h, p]
 *   out     = y, or y * z * sigmoid(z) with a gate z
 *
 * from the slot's state when has_initial[b] != 0, else from zero; the state after the last
 * token goes to the slot (an empty sequence leaves its slot as it is, or zeroed without
 * has_initial). The state is held in 32 bits. A[h] <= 0 is expected of a decay; the recurrent
 * kernel takes any A, the chunked one any A for which no chunk's growth overflows.
 *
 * Routes: the recurrent kernel walks the tokens one by one and takes every size it can hold
 * (K <= 256); the chunked kernel takes 128 tokens at a time as matrix products on the tensor
 * cores (P % 8 == 0, K % 8 == 0, K <= 128, rows on 16-byte boundaries). AUTO picks by size: the chunked kernel where it
 * serves and the sequences have 16 tokens or more on average. Token by token a prompt takes 0.7 us a token with
 * 128 states and 1.7 with 256, however few heads there are, so long prompts of more than 128 states, or off those boundaries, are
 * slow: 8 x 4096 tokens of 64 heads x 64 channels take 20 ms with 256 states, 0.5 ms with 128.
 *
 * Precision: both routes compute in 32 bits and round an output once. The chunked kernel's matrix products take their
 * factors as sums of BF16 terms: three (24 bits) in what is added to the state, two (16 bits, 2^-16 of a term)
 * in the outputs, whose own rounding is 2^-9.
 *
 * NaN and infinities reach what depends on them by the formula and nothing else. Token by token the results are
 * the formula's; the chunked kernel may give NaN where the formula gives an infinity.
 */
typedef enum ccu_scan_route {
  CCU_SCAN_AUTO = 0,
  CCU_SCAN_RECURRENT = 1,
  CCU_SCAN_CHUNKED = 2,
  CCU_SCAN_ROUTE_COUNT = 3
} ccu_scan_route_t;

typedef struct ccu_selective_scan_args {
  const void *x;              /* BF16 [T, H, P], unit stride along P */
  int64_t x_stride_t, x_stride_h;
  const void *dt;             /* BF16 [T, H], unit stride along H */
  int64_t dt_stride_t;
  const void *b;              /* BF16 [T, G, K], unit stride along K */
  int64_t b_stride_t, b_stride_g;
  const void *c;              /* BF16 [T, G, K], unit stride along K */
  int64_t c_stride_t, c_stride_g;
  const void *z;              /* BF16 [T, H, P] or NULL, unit stride along P */
  int64_t z_stride_t, z_stride_h;
  const float *A;             /* FP32 [H] */
  const float *D;             /* FP32 [H] or NULL */
  const float *dt_bias;       /* FP32 [H] or NULL */
  const int32_t *cu_seqlens;  /* int32 [n_seq + 1] */
  const int32_t *indices;     /* int32 [n_seq] or NULL */
  const int32_t *has_initial; /* int32 [n_seq] or NULL */
  float *state;               /* FP32 [S, H, P, K], a slot contiguous, slots stride_s apart */
  int64_t state_stride_s;
  void *out;                  /* BF16 [T, H, P], unit stride along P; must not overlap an input */
  int64_t out_stride_t, out_stride_h;
  void *workspace;            /* device scratch, 16-byte aligned; see ..._workspace_bytes */
  int64_t workspace_bytes;
  int32_t *status_dev;        /* device word for CCU_DEVERR_*, or NULL */
  int64_t T, n_seq, H, P, K, G, S;
  int32_t dt_softplus;        /* nonzero: softplus */
  int32_t route;              /* ccu_scan_route_t */
} ccu_selective_scan_args_t;

CCU_API ccu_status_t ccu_selective_scan(const ccu_selective_scan_args_t *args, ccu_stream_t stream);

/* Bytes of workspace ccu_selective_scan needs for these arguments on the current device (0: none);
 * -1 for arguments it declines. Pointers other than NULL-ness and alignment do not matter. */
CCU_API int64_t ccu_selective_scan_workspace_bytes(const ccu_selective_scan_args_t *args);

/* The kernel a call with these arguments takes (a ccu_scan_route_t), or -1 for arguments the
 * call declines. Makes no CUDA call. */
CCU_API int32_t ccu_selective_scan_select_route(const ccu_selective_scan_args_t *args);

/*
 * ccu_selective_state_update -- one token per row: the convolution step and the state step,
 * both in place on the row's cache slot.
 *
 * xbc[n] holds the H * P channels of x, then G * K of B, then G * K of C. With conv_weight they
 * first go through the convolution step of ccu_conv1d_update (linear state; the sums and the
 * activation stay in 32 bits, they are not rounded to BF16 in between), without it they are
 * taken as they are and conv_state, conv_bias and act are ignored. Then one step of the recurrence of
 * ccu_selective_scan.
 */
typedef struct ccu_selective_state_update_args {
  const void *xbc;            /* BF16 [N, H*P + 2*G*K], row stride ld_xbc */
  int64_t ld_xbc;
  const void *conv_weight;    /* BF16 contiguous [H*P + 2*G*K, W], or NULL: no convolution */
  const void *conv_bias;      /* BF16 [H*P + 2*G*K] or NULL */
  void *conv_state;           /* BF16 [S, H*P + 2*G*K, L] by strides */
  int64_t conv_stride_s, conv_stride_d, conv_stride_l;
  const void *dt;             /* BF16 [N, H], unit stride along H */
  int64_t dt_stride_n;
  const void *z;              /* BF16 [N, H, P] or NULL, unit stride along P */
  int64_t z_stride_n, z_stride_h;
  const float *A;             /* FP32 [H] */
  const float *D;             /* FP32 [H] or NULL */
  const float *dt_bias;       /* FP32 [H] or NULL */
  const int32_t *indices;     /* int32 [N] or NULL */
  float *state;               /* FP32 [S, H, P, K], a slot contiguous, slots stride_s apart */
  int64_t state_stride_s;
  void *out;                  /* BF16 [N, H, P], unit stride along P; must not overlap an input */
  int64_t out_stride_n, out_stride_h;
  void *workspace;            /* device scratch, 16-byte aligned: 4 * N * (H*P + 2*G*K) bytes
                                 with conv_weight, else unused */
  int64_t workspace_bytes;
  int32_t *status_dev;        /* device word for CCU_DEVERR_RANGE, or NULL */
  int64_t N, H, P, K, G, S, L, W; /* W >= 1, L >= max(W - 1, 1) with conv_weight; K <= 256 */
  int32_t act;                /* ccu_act_t of the convolution */
  int32_t dt_softplus;        /* nonzero: softplus */
} ccu_selective_state_update_args_t;

CCU_API ccu_status_t ccu_selective_state_update(const ccu_selective_state_update_args_t *args,
                                                ccu_stream_t stream);

/* Bytes of workspace ccu_selective_state_update needs; -1 for negative sizes. */
CCU_API int64_t ccu_selective_state_update_workspace_bytes(int64_t N, int64_t H, int64_t P, int64_t K,
                                                           int64_t G, int32_t has_conv);

/*
 * ccu_w4_matmul -- products of a few rows with a matrix of 4-bit weights.
 *
 *   out[m, o] = sum_i x[m, i] * (q[o, i] - zero[o, i / group]) * scale[o, i / group]
 *
 * with q[o, i] in 0..15 stored two a byte (even i in the low half) and zero = 8 when zeros is
 * NULL. Products are exact, sums are held in 32 bits, out is rounded once. An infinite or NaN x gives what the
 * formula gives, for operands on any boundary. Meant for the token
 * rows of a decode step; any M works, the weights are read once for every 64 rows (32 with groups of 32).
 */
typedef struct ccu_w4_matmul_args {
  const void *x;       /* BF16 [M, I], row stride ld_x */
  int64_t ld_x;
  const void *qweight; /* bytes, contiguous [O, I / 2], 4-byte aligned */
  const void *scales;  /* BF16 contiguous [O, I / group] */
  const void *zeros;   /* BF16 contiguous [O, I / group] or NULL */
  void *out;           /* BF16 [M, O], row stride ld_out; must not overlap an input */
  int64_t ld_out;
  int64_t M, I, O;
  int64_t group;       /* 32, 64 or 128; I % group == 0 */
} ccu_w4_matmul_args_t;

CCU_API ccu_status_t ccu_w4_matmul(const ccu_w4_matmul_args_t *args, ccu_stream_t stream);

/*
 * ccu_gated_delta_rule -- the gated delta rule over packed prompts.
 *
 * Per head h (its group g = h / (H / G)) a matrix state s[P, K] runs over the tokens of a
 * sequence:
 *
 *   decay   = exp(A[h] * softplus(a[t, h] + dt_bias[h])),   beta = sigmoid(b[t, h])
 *   kn, qn  = k[t, g] / sqrt(|k[t, g]|^2 + 1e-6), q alike    (k and q as they are when qk_norm is 0)
 *   s[p, k] = decay * s[p, k]
 *   u[p]    = beta * (v[t, h, p] - sum_k s[p, k] * kn[k])
 *   s[p, k] = s[p, k] + u[p] * kn[k]
 *   out[p]  = scale * sum_k s[p, k] * qn[k]
 *
 * from the slot's state when has_initial[b] != 0, else from zero; the state after the last
 * token goes to the slot (an empty sequence leaves its slot as it is, or zeroed without
 * has_initial). The state is held in 32 bits, and so is everything that goes into it; an output is rounded once. The squares
 * of a row are summed in 32 bits: entries above 1e18 make an infinite norm, and a row of zeros. A[h] <= 0 is expected of a decay.
 * Rows of `out` outside every sequence are left as they were; a padding sequence (slot -1) has outputs of +0 and no state. Two sequences
 * of a call must not share a slot.
 *
 * Two kernels (route, as in ccu_selective_scan). CCU_SCAN_RECURRENT goes token by token and serves every size. CCU_SCAN_CHUNKED takes 64
 * tokens at a time on the tensor cores: P and K in multiples of 8, K <= 128, and q, k, v, out, their rows and heads, state and its slots on
 * 16-byte boundaries, with no stride of 0 along more than one entry; others are declined with CCU_ERR_NOT_IMPLEMENTED. The factors of its products carry 24 bits each, in
 * the state and in the outputs. CCU_SCAN_AUTO takes it where it serves and sequences average 16 tokens (with P < 128, 16 * 128 / P). Sequences
 * much longer than that with few heads are cut into segments that run side by side, and where sequences times heads are somewhat more than the SMs (or
 * twice, three times as many) some are cut in two; both need the workspace.
 *
 * NaN and infinities reach what depends on them by the formula and nothing else; they reach no earlier token. The chunked kernel
 * gives NaN from its token on where v (its channel), k (all channels) or a key's sum of squares is infinite, and without qk_norm expects
 * keys that keep the rule from overflowing within 64 tokens (|k| about 1): where it does, the outputs of those 64 may all be NaN.
 */
typedef struct ccu_gated_delta_rule_args {
  const void *q;              /* BF16 [T, G, K], unit stride along K */
  int64_t q_stride_t, q_stride_g;
  const void *k;              /* BF16 [T, G, K], unit stride along K */
  int64_t k_stride_t, k_stride_g;
  const void *v;              /* BF16 [T, H, P], unit stride along P */
  int64_t v_stride_t, v_stride_h;
  const void *a;              /* BF16 [T, H], unit stride along H */
  int64_t a_stride_t;
  const void *b;              /* BF16 [T, H], unit stride along H */
  int64_t b_stride_t;
  const float *A;             /* FP32 [H] */
  const float *dt_bias;       /* FP32 [H] or NULL */
  const int32_t *cu_seqlens;  /* int32 [n_seq + 1] */
  const int32_t *indices;     /* int32 [n_seq] or NULL */
  const int32_t *has_initial; /* int32 [n_seq] or NULL */
  float *state;               /* FP32 [S, H, P, K], a slot contiguous, slots stride_s apart */
  int64_t state_stride_s;
  void *out;                  /* BF16 [T, H, P], unit stride along P; must not overlap an input */
  int64_t out_stride_t, out_stride_h;
  void *workspace;            /* device scratch, 16-byte aligned; see ..._workspace_bytes */
  int64_t workspace_bytes;
  int32_t *status_dev;        /* device word for CCU_DEVERR_*, or NULL */
  int64_t T, n_seq, H, P, K, G, S; /* K <= 256 */
  float scale;                /* 0: 1 / sqrt(K) */
  int32_t qk_norm;            /* nonzero: q and k are brought to unit length */
  int32_t route;              /* ccu_scan_route_t */
  int32_t reserved;           /* 0 */
} ccu_gated_delta_rule_args_t;

CCU_API ccu_status_t ccu_gated_delta_rule(const ccu_gated_delta_rule_args_t *args, ccu_stream_t stream);

/* Bytes of workspace ccu_gated_delta_rule needs for these arguments on the current device (0: none);
 * -1 for arguments it declines. Pointers other than NULL-ness and alignment do not matter. */
CCU_API int64_t ccu_gated_delta_rule_workspace_bytes(const ccu_gated_delta_rule_args_t *args);

/* The kernel a call with these arguments takes (a ccu_scan_route_t), or -1 for arguments the
 * call declines. Makes no CUDA call. */
CCU_API int32_t ccu_gated_delta_rule_select_route(const ccu_gated_delta_rule_args_t *args);

/*
 * ccu_gated_delta_update -- one token per row: the convolution step and the state step of the gated delta rule,
 * both in place on the row's cache slot.
 *
 * qkv[n] holds the G * K channels of q, then G * K of k, then H * P of v. With conv_weight they go through the
 * convolution step first, as in ccu_selective_state_update but for the SiLU, which is that of 32 bits here too; then one step of the recurrence of ccu_gated_delta_rule. Two rows
 * of a call must not share a slot.
 */
typedef struct ccu_gated_delta_update_args {
  const void *qkv;            /* BF16 [N, 2*G*K + H*P], row stride ld_qkv */
  int64_t ld_qkv;
  const void *conv_weight;    /* BF16 contiguous [2*G*K + H*P, W], or NULL: no convolution */
  const void *conv_bias;      /* BF16 [2*G*K + H*P] or NULL */
  void *conv_state;           /* BF16 [S, 2*G*K + H*P, L] by strides */
  int64_t conv_stride_s, conv_stride_d, conv_stride_l;
  const void *a;              /* BF16 [N, H], unit stride along H */
  int64_t a_stride_n;
  const void *b;              /* BF16 [N, H], unit stride along H */
  int64_t b_stride_n;
  const float *A;             /* FP32 [H] */
  const float *dt_bias;       /* FP32 [H] or NULL */
  const int32_t *indices;     /* int32 [N] or NULL */
  float *state;               /* FP32 [S, H, P, K], a slot contiguous, slots stride_s apart */
  int64_t state_stride_s;
  void *out;                  /* BF16 [N, H, P], unit stride along P; must not overlap an input */
  int64_t out_stride_n, out_stride_h;
  void *workspace;            /* device scratch, 16-byte aligned: 4 * N * (2*G*K + H*P) bytes
                                 with conv_weight, else unused */
  int64_t workspace_bytes;
  int32_t *status_dev;        /* device word for CCU_DEVERR_RANGE, or NULL */
  int64_t N, H, P, K, G, S, L, W; /* W >= 1, L >= max(W - 1, 1) with conv_weight; K <= 256 */
  float scale;                /* 0: 1 / sqrt(K) */
  int32_t qk_norm;            /* nonzero: q and k are brought to unit length */
  int32_t act;                /* ccu_act_t of the convolution */
  int32_t reserved;           /* 0 */
} ccu_gated_delta_update_args_t;

CCU_API ccu_status_t ccu_gated_delta_update(const ccu_gated_delta_update_args_t *args, ccu_stream_t stream);

/* Bytes of workspace ccu_gated_delta_update needs; -1 for negative sizes. */
CCU_API int64_t ccu_gated_delta_update_workspace_bytes(int64_t N, int64_t H, int64_t P, int64_t K,
                                                       int64_t G, int32_t has_conv);

/* Type of a tensor that may be either. */
typedef enum ccu_dtype {
  CCU_DTYPE_BF16 = 0,
  CCU_DTYPE_FP32 = 1
} ccu_dtype_t;

/*
 * ccu_gated_rms_norm -- the norm behind a recurrence, with its gate. Per token t and head (or group of channels) h:
 *
 *   out = y / sqrt(mean(y^2) + eps) * weight * g        y = x,   g = z * sigmoid(z)      (1 without z)
 *   out = y / sqrt(mean(y^2) + eps) * weight            y = x * z * sigmoid(z)           with gate_first
 *
 * over the P entries of x[t, h]. Computed in 32 bits, rounded once.
 */
typedef struct ccu_gated_rms_norm_args {
  const void *x;              /* BF16 [T, H, P], unit stride along P */
  int64_t x_stride_t, x_stride_h;
  const void *z;              /* BF16 [T, H, P] or NULL, unit stride along P */
  int64_t z_stride_t, z_stride_h;
  const void *weight;         /* [P], or [H, P] with weight_stride_h, or NULL (1) */
  int64_t weight_stride_h;    /* 0: one weight for all heads */
  void *out;                  /* BF16 [T, H, P], unit stride along P; must not overlap an input */
  int64_t out_stride_t, out_stride_h;
  int64_t T, H, P;
  float eps;
  int32_t gate_first;         /* nonzero: the gated x is normed */
  int32_t weight_type;        /* ccu_dtype_t */
  int32_t reserved;           /* 0 */
} ccu_gated_rms_norm_args_t;

CCU_API ccu_status_t ccu_gated_rms_norm(const ccu_gated_rms_norm_args_t *args, ccu_stream_t stream);

/*
 * ccu_residual_rms_norm -- between two blocks: what the last one gave is normed (with post_weight), scaled and added to the
 * residual, which is normed for the next one. Per row t:
 *
 *   y        = x, or x / sqrt(mean(x^2) + eps) * post_weight
 *   residual = residual + scale * y                                    in place
 *   out      = residual / sqrt(mean(residual^2) + eps) * weight
 *
 * over the D entries of a row. Computed in 32 bits; the sum goes into the norm as it is and is rounded to the residual's
 * type where it is stored.
 */
typedef struct ccu_residual_rms_norm_args {
  const void *x;              /* BF16 [T, D], row stride ld_x, unit stride along D */
  int64_t ld_x;
  void *residual;             /* [T, D], row stride ld_residual, unit stride along D; must not overlap another tensor */
  int64_t ld_residual;
  const void *weight;         /* [D] or NULL (1) */
  const void *post_weight;    /* [D] or NULL: x is not normed; of weight's type */
  void *out;                  /* BF16 [T, D], row stride ld_out; must not overlap an input */
  int64_t ld_out;
  int64_t T, D;
  float scale, eps;           /* a scale of 0 adds nothing: there is no default */
  int32_t residual_type;      /* ccu_dtype_t */
  int32_t weight_type;        /* ccu_dtype_t */
} ccu_residual_rms_norm_args_t;

CCU_API ccu_status_t ccu_residual_rms_norm(const ccu_residual_rms_norm_args_t *args, ccu_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CCU_SSM_H */

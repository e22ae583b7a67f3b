/*
 * muon.h -- C ABI of the MI355X (gfx950) Muon optimizer step, and of the layer
 * operators that make the gradients it takes (layer norm, the linear layer's
 * products, 8-bit activation checkpoints; see "the layer operators" below; the
 * gated feed-forward, norms around a block and dropout; see "the block operators").
 *
 * One muon_step call performs, for every 2-D weight in a list, the Muon step the speedrun
 * pages describe:
 *
 *   m'  = beta * m + g                      momentum, no dampening
 *   u   = g + beta * m'  (Nesterov)  or  m'
 *   X0  = u / (||u||_F + eps),  transposed when rows > cols
 *   ns_steps x { A = X X^T ; B = b A + c A A ; X = a X + B X }
 *   O   = X (transposed back)
 *   W'  = W * (1 - lr * wd) - lr * sqrt(max(1, rows/cols)) * O
 *
 * Sources: "14 -- modded-nanogpt: the Speedrun Community", section 3 "Muon"
 * (pseudocode: momentum form, update sign, 5 iterations); "NanoGPT Speedrun"
 * (modded-nanogpt README mirror), Muon section (the Newton-Schulz routine:
 * eps = 1e-7 on the Frobenius norm, the transpose rule, coefficients
 * (3.4445, -4.7750, 2.0315); the practices list: Nesterov momentum, bfloat16
 * execution); same README, GPT-2 medium track ("standard weight decay").
 * Readings where the pages are silent: the Nesterov form u = g + beta m', the
 * decoupled lr-coupled decay on the old W, and the shape scale.
 *
 * Conventions shared by every entry point
 *   - Matrices are row-major: element (i, j) at ptr[i * ld + j]; ld counts
 *     elements and must be >= cols.
 *   - Every data pointer is a device pointer on the handle's device, owned by
 *     the caller, and must stay valid until the stream has passed the work.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream) and
 *     the call returns without synchronising (except the first call of a new
 *     signature, which waits for its plan upload).  The handle's workspaces
 *     are shared by its calls: calls on one handle must be ordered on one
 *     stream (or externally).
 *   - Validation happens before anything is enqueued; a call that returns an
 *     error enqueued nothing and changed no caller memory.
 *   - NaN/Inf inputs are not checked; they propagate within their matrix.
 *   - A handle is bound to one device and is not thread-safe; distinct handles
 *     are independent.
 */
#ifndef MUON_MI355X_H
#define MUON_MI355X_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_ABI_VERSION 8

typedef enum muon_status {
    MUON_OK = 0,
    MUON_ERR_INVALID_ARG = 1,  /* null pointer, bad size/ld, aliasing, bad ns_steps */
    MUON_ERR_DTYPE = 2,        /* unknown storage dtype or compute mode */
    MUON_ERR_NO_DEVICE = 3,    /* no HIP device, or the handle's device is gone */
    MUON_ERR_OOM = 4,          /* workspace allocation failed */
    MUON_ERR_HIP = 5           /* a HIP runtime call or launch failed; see muon_last_error */
} muon_status;

typedef enum muon_dtype {
    MUON_BF16 = 0,             /* bfloat16 storage */
    MUON_F32 = 1               /* float32 storage */
} muon_dtype;

typedef enum muon_compute {
    MUON_COMPUTE_BF16 = 0,     /* bf16 MFMA operands, fp32 accumulation; X kept between iterations
                                  to ~16 bits (bf16 copy + 8-bit remainder), A and B in bf16.
                                  Matrices (or blocks) with min(rows, cols) <= 64 run the iteration
                                  in fp32 in this mode too: their products cost next to nothing and
                                  bf16 operands cost them the most accuracy */
    MUON_COMPUTE_FP32 = 1      /* fp32 MFMA operands and storage: validation mode */
} muon_compute;

/* init flags */
#define MUON_INIT_PROFILE     0x1u   /* time kernel launches with HIP events (all roles, or see below) */
#define MUON_INIT_FAIL_ALLOC  0x2u   /* test hook: every workspace allocation fails (MUON_ERR_OOM) */
#define MUON_INIT_DEBUG       0x4u   /* debug checks: a guard band of a fixed pattern after every workspace
                                        buffer of muon_step's plans, checked after every step (which then
                                        waits for its stream); an overwritten band fails the call with
                                        MUON_ERR_HIP and the count of damaged words in muon_last_error */

/* Kernel roles, as named in muon_kernel_stats.name. */
typedef enum muon_role {
    MUON_ROLE_MOMENTUM = 0,    /* "momentum_norm" */
    MUON_ROLE_FINALIZE = 1,    /* "norm_finalize" */
    MUON_ROLE_GRAM = 2,        /* "ns_gram" */
    MUON_ROLE_POLY = 3,        /* "ns_poly" */
    MUON_ROLE_AXPY = 4,        /* "ns_axpy" (every iteration but the last) */
    MUON_ROLE_AXPY_UPDATE = 5, /* "ns_axpy_update" (last iteration and the weight update) */
    MUON_ROLE_DIRECT = 6,      /* "direct_update" (ns_steps == 0) */
    MUON_ROLE_FILL = 7,        /* "fill_zero" (workspace initialisation) */
    MUON_ROLE_ADAMW = 8,       /* "adamw" */
    MUON_ROLE_RESCALE = 9      /* "norm_rescale" (operand copy of inputs with an extreme norm) */
} muon_role;

/* With MUON_INIT_PROFILE, time only the roles whose bits are set in `mask`
 * (bit r = role r); no bits = every role.  Each timed launch carries its own
 * start/stop events, which costs a little time per launch. */
#define MUON_INIT_PROFILE_ROLES(mask) ((((uint32_t)(mask)) & 0x3FFu) << 16)

/* One weight matrix of the list handed to muon_step. */
typedef struct muon_matrix {
    void       *param;         /* rows x cols, `dtype`, updated in place */
    const void *grad;          /* rows x cols, `dtype`, read only */
    float      *momentum;      /* rows x cols float32, updated in place (start at 0) */
    float      *update_out;    /* optional rows x cols float32: receives O (validation); may be NULL */
    int64_t     rows, cols;    /* stored shape, both >= 1 */
    int64_t     ld_param, ld_grad, ld_mom, ld_update;   /* leading dims, elements, >= cols */
    int32_t     dtype;         /* muon_dtype of param and grad */
    int32_t     block_rows;    /* sub-block orthogonalisation: the matrix is cut into   */
    int32_t     block_cols;    /* block_rows x block_cols blocks (0 = the whole dimension;
                                  each must divide its dimension), and every block is a
                                  matrix of its own for the norm, the transpose rule, the
                                  iteration and the shape scale, as when query and key
                                  weights are orthogonalised in pairs of heads ("NanoGPT
                                  Speedrun", record list).  Momentum is elementwise and
                                  unaffected.  0, 0 = the plain step. */
    int32_t     reserved;      /* must be 0 */
} muon_matrix;

/* Hyperparameters, shared by every matrix of one call. */
typedef struct muon_hparams {
    float   lr;                /* learning rate */
    float   beta;              /* momentum, 0.95 on the pages */
    float   weight_decay;      /* decoupled: W *= 1 - lr * weight_decay */
    float   eps;               /* added to the Frobenius norm, 1e-7 on the pages */
    float   a, b, c;           /* quintic coefficients, (3.4445, -4.7750, 2.0315); finite, a != 0 */
    int32_t nesterov;          /* 0 or 1 */
    int32_t ns_steps;          /* 0..64; 5 on the pages */
    int32_t compute;           /* muon_compute */
    const float *coeffs;       /* optional host array of ns_steps triples (a_k, b_k, c_k), iteration k
                                  using the k-th in place of (a, b, c): per-iteration schedules such as
                                  Polar Express, named in the record list of "NanoGPT Speedrun"
                                  (modded-nanogpt README mirror); each finite, a_k != 0.  Read during
                                  the call only.  NULL = (a, b, c) for every iteration. */
} muon_hparams;

typedef struct muon_handle muon_handle;

/* Per-kernel launch statistics gathered when the handle was created with MUON_INIT_PROFILE. */
typedef struct muon_kernel_stats {
    char    name[48];          /* kernel role: "momentum_norm", "ns_gram", ... */
    int64_t launches;          /* completed launches timed */
    double  total_ms;          /* summed HIP-event durations */
} muon_kernel_stats;

/* One tensor of the list handed to muon_adamw_step: any parameter Muon does not
 * take (embeddings, output head, norm gains, biases), as `numel` contiguous
 * elements. */
typedef struct muon_adamw_tensor {
    void       *param;         /* numel elements, `dtype`, updated in place */
    const void *grad;          /* numel elements, `dtype`, read only */
    float      *exp_avg;       /* numel float32, first moment, updated in place (start at 0) */
    float      *exp_avg_sq;    /* numel float32, second moment, updated in place (start at 0) */
    int64_t     numel;         /* >= 0; 0 = nothing to do for this entry */
    int32_t     dtype;         /* muon_dtype of param and grad */
    int32_t     reserved;      /* must be 0 */
} muon_adamw_tensor;

/* AdamW hyperparameters, shared by every tensor of one call. */
typedef struct muon_adamw_hparams {
    float   lr;                /* learning rate, finite */
    float   beta1, beta2;      /* moment decays, each in [0, 1) */
    float   eps;               /* added to sqrt of the corrected second moment, finite, > 0 */
    float   weight_decay;      /* decoupled: p *= 1 - lr * weight_decay, finite */
    int32_t step;              /* 1-based step count t of this update (bias corrections 1 - beta^t) */
} muon_adamw_hparams;

/* ---- the layer operators: what makes the gradients the steps above take ---- */

/* 8-bit activation checkpoint of a rows x cols matrix.  The 32 columns
 * [32 j, 32 j + 32) of a row (fewer at its end) form a group that shares one
 * exponent byte: element (r, c) stands for
 *
 *   codes[r * ld_codes + c] * 2^(exponents[r * ld_exponents + c / 32] - 127).
 *
 * The encoder takes the smallest power of two, not under 2^-126, that keeps
 * every code of the group within -127..127, and rounds to nearest even: an
 * element is off by at most half a step, 1/127 of its group's largest magnitude
 * (1/254 at best), or, in a group under 63.5 * 2^-126, 2^-127.  Decoding is
 * exact in bfloat16 and float32.  A group holding an infinity or a NaN gets
 * exponent byte 255 and codes 0: all of it decodes to NaN.  The encoder writes
 * bytes 1..249 and 255; byte 0 decodes to zeros. */
typedef struct muon_act8 {
    int8_t  *codes;            /* rows x cols */
    uint8_t *exponents;        /* rows x ceil(cols / 32) */
    int64_t  ld_codes;         /* >= cols */
    int64_t  ld_exponents;     /* >= ceil(cols / 32) */
} muon_act8;
#define MUON_ACT8_GROUP 32

typedef enum muon_activation {
    MUON_ACT_NONE = 0,
    MUON_ACT_GELU = 1,         /* 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)));
                                  at infinite z the limits: 0 and infinity, derivatives 0 and 1 */
    MUON_ACT_RELU_SQ = 2       /* max(z, 0)^2 */
} muon_activation;

/* How a linear layer's weight is stored; either is a muon_matrix for muon_step. */
typedef enum muon_weight_layout {
    MUON_W_IN_OUT = 0,         /* in x out */
    MUON_W_OUT_IN = 1          /* out x in */
} muon_weight_layout;

/* Arguments of muon_layernorm_forward.  Pointers noted "optional" may be NULL. */
typedef struct muon_layernorm_args {
    const void *x;             /* rows x cols, `dtype` */
    const void *gain;          /* cols, `param_dtype` */
    const void *bias;          /* cols, `param_dtype`; optional */
    void       *y;             /* rows x cols, `dtype` */
    float      *mean;          /* rows; optional */
    float      *rstd;          /* rows; optional */
    muon_act8   y8;            /* y's 8-bit checkpoint, of y before its rounding; codes NULL = none */
    int64_t     rows, cols;    /* rows >= 0, 1 <= cols <= 2^20 */
    int64_t     ld_x, ld_y;
    int32_t     dtype, param_dtype;   /* muon_dtype */
    float       eps;           /* added to the variance, >= 0, finite */
    int32_t     reserved;      /* must be 0 */
} muon_layernorm_args;

/* Arguments of muon_layernorm_backward. */
typedef struct muon_layernorm_grad_args {
    const void  *dy;           /* rows x cols, `dtype` */
    const void  *x;            /* rows x cols, `dtype`: the forward pass's input */
    const void  *gain;         /* cols, `param_dtype` */
    const float *mean, *rstd;  /* rows: as the forward pass wrote them */
    const void  *add;          /* rows x cols, `dtype`, added to dx (the residual path's gradient); optional;
                                  may be dx itself (same leading dimension) */
    void        *dx;           /* rows x cols, `dtype` */
    void        *dgain;        /* cols, `param_dtype` */
    void        *dbias;        /* cols, `param_dtype`; optional */
    int64_t      rows, cols;
    int64_t      ld_dy, ld_x, ld_add, ld_dx;
    int32_t      dtype, param_dtype;
    int32_t      accumulate;   /* 1: dgain and dbias are added to */
    int32_t      reserved;     /* must be 0 */
} muon_layernorm_grad_args;

/* Arguments of muon_linear_forward. */
typedef struct muon_linear_args {
    const void *x;             /* rows x in, `dtype` */
    const void *w;             /* in x out or out x in (w_layout), `dtype` */
    const void *bias;          /* out, `bias_dtype`; optional */
    const void *residual;      /* rows x out, `dtype`, added after the activation; optional; may be y itself */
    void       *y;             /* rows x out, `dtype` */
    void       *z;             /* rows x out, `dtype`: receives x W + bias; optional */
    muon_act8   z8;            /* or its 8-bit checkpoint, taken before any rounding; codes NULL = none */
    int64_t     rows, in, out; /* rows >= 0; 1 <= in, out <= 2^20 */
    int64_t     ld_x, ld_w, ld_residual, ld_y, ld_z;
    int32_t     dtype, bias_dtype;    /* muon_dtype */
    int32_t     activation;    /* muon_activation */
    int32_t     w_layout;      /* muon_weight_layout */
    int32_t     reserved;      /* must be 0 */
} muon_linear_args;

/* Arguments of muon_linear_grad_input. */
typedef struct muon_linear_grad_input_args {
    const void *dy;            /* rows x out, `dtype` */
    const void *w;             /* as in the forward pass */
    const void *z;             /* rows x in, `dtype`: the pre-activation behind this layer's input; optional */
    muon_act8   z8;            /* or its 8-bit checkpoint (read); codes NULL = none */
    const void *add;           /* rows x in, `dtype`, added last; optional; may be dx itself */
    void       *dx;            /* rows x in, `dtype` */
    void       *act_out;       /* rows x in, `dtype`: receives act(z), this layer's input; optional, needs z or z8 */
    int64_t     rows, in, out;
    int64_t     ld_dy, ld_w, ld_z, ld_add, ld_dx, ld_act_out;
    int32_t     dtype;
    int32_t     activation;    /* of z; MUON_ACT_NONE without z and z8 */
    int32_t     w_layout;
    int32_t     reserved;      /* must be 0 */
} muon_linear_grad_input_args;

/* Arguments of muon_linear_grad_weight. */
typedef struct muon_linear_grad_weight_args {
    const void *x;             /* rows x in, `dtype`; or NULL and */
    muon_act8   x8;            /* its 8-bit checkpoint (read) */
    const void *dy;            /* rows x out, `dtype` */
    void       *dw;            /* in x out or out x in (w_layout), `dw_dtype` */
    void       *db;            /* out, `db_dtype`; optional */
    int64_t     rows, in, out;
    int64_t     ld_x, ld_dy, ld_dw;
    int32_t     dtype, dw_dtype, db_dtype;
    int32_t     w_layout;
    int32_t     accumulate;    /* 1: dw and db are added to */
    int32_t     reserved;      /* must be 0 */
} muon_linear_grad_weight_args;

/* ---- the block operators: a gated feed-forward block and what stands around it ---- */

/* The gate's activation, act(z); at infinite z the limits, forward and backward. */
typedef enum muon_gate {
    MUON_GATE_SILU = 0,        /* z / (1 + exp(-z)) */
    MUON_GATE_GELU = 1,        /* as MUON_ACT_GELU */
    MUON_GATE_SIGMOID = 2,     /* 1 / (1 + exp(-z)) */
    MUON_GATE_RELU = 3         /* max(z, 0) */
} muon_gate;

/* Arguments of muon_gated_forward.  The two tensors of a pair have one leading
 * dimension; a weight that holds both projections is two such views of it. */
typedef struct muon_gated_args {
    const void *x;             /* rows x in, `dtype` */
    const void *w_gate, *w_up; /* in x hidden or hidden x in (w_layout), `dtype` */
    const void *bias_gate, *bias_up;   /* hidden, `bias_dtype`; each optional */
    void       *h;             /* rows x hidden, `dtype` */
    void       *gate, *up;     /* rows x hidden, `dtype`: receive both pre-activations; both or neither */
    muon_act8   gate8, up8;    /* or their 8-bit checkpoints, taken before any rounding */
    int64_t     rows, in, hidden;      /* rows >= 0; 1 <= in, hidden <= 2^20 */
    int64_t     ld_x, ld_w, ld_h, ld_z;    /* ld_z: of gate and up */
    int32_t     dtype, bias_dtype;     /* muon_dtype */
    int32_t     activation;    /* muon_gate */
    int32_t     w_layout;      /* muon_weight_layout */
    int32_t     reserved;      /* must be 0 */
} muon_gated_args;

/* Arguments of muon_gated_grad_hidden. */
typedef struct muon_gated_grad_hidden_args {
    const void *dy;            /* rows x out, `dtype`: the gradient behind the down projection */
    const void *w_down;        /* hidden x out or out x hidden (w_layout), `dtype` */
    const void *gate, *up;     /* rows x hidden, `dtype`: both pre-activations, or NULL and */
    muon_act8   gate8, up8;    /* their 8-bit checkpoints (read) */
    void       *dgate, *dup;   /* rows x hidden, `dtype` */
    void       *h;             /* rows x hidden, `dtype`: receives act(gate) up; optional */
    int64_t     rows, hidden, out;
    int64_t     ld_dy, ld_w, ld_z, ld_dz, ld_h;    /* ld_z: of gate and up; ld_dz: of dgate and dup */
    int32_t     dtype;
    int32_t     activation;    /* muon_gate */
    int32_t     w_layout;
    int32_t     reserved;      /* must be 0 */
} muon_gated_grad_hidden_args;

/* Arguments of muon_gated_grad_input. */
typedef struct muon_gated_grad_input_args {
    const void *dgate, *dup;   /* rows x hidden, `dtype` */
    const void *w_gate, *w_up; /* as in the forward pass */
    const void *add;           /* rows x in, `dtype`, added last; optional; may be dx itself */
    void       *dx;            /* rows x in, `dtype` */
    int64_t     rows, in, hidden;
    int64_t     ld_dz, ld_w, ld_add, ld_dx;
    int32_t     dtype;
    int32_t     w_layout;
    int32_t     reserved;      /* must be 0 */
} muon_gated_grad_input_args;

/* Arguments of muon_gated_grad_weight. */
typedef struct muon_gated_grad_weight_args {
    const void *x;             /* rows x in, `dtype`; or NULL and */
    muon_act8   x8;            /* its 8-bit checkpoint (read) */
    const void *dgate, *dup;   /* rows x hidden, `dtype` */
    void       *dw_gate, *dw_up;       /* in x hidden or hidden x in (w_layout), `dw_dtype` */
    void       *db_gate, *db_up;       /* hidden, `db_dtype`; each optional */
    int64_t     rows, in, hidden;
    int64_t     ld_x, ld_dz, ld_dw;
    int32_t     dtype, dw_dtype, db_dtype;
    int32_t     w_layout;
    int32_t     accumulate;    /* 1: the four outputs are added to */
    int32_t     reserved;      /* must be 0 */
} muon_gated_grad_weight_args;

/* A dropout mask.  Nothing of it is stored: element (r, c) of a matrix takes 16
 * bits of a counter-based generator, Philox 4x32 of ten rounds (Salmon, Moraes,
 * Dror and Shaw 2011), with the key (seed mod 2^32, seed / 2^32) and the counter
 * (c / 8, r, n mod 2^32, n / 2^32), n = offset (+ *step) mod 2^64: half c mod 2
 * (0: the low one) of word (c / 2) mod 4.  With T = p * 65536 rounded to nearest
 * (halves to even), an element whose bits are under T is dropped, and becomes 0
 * whatever it was; the others are multiplied by 65536 / (65536 - T).  So a mask
 * depends on the element's place in its matrix alone, and the same seed and
 * offset give it again, forward and backward.  Give every use of a step its own
 * offset, or its own seed. */
typedef struct muon_dropout_mask {
    float     p;               /* 0 <= p <= 1 */
    int32_t   reserved;        /* must be 0 */
    uint64_t  seed, offset;
    const uint64_t *step;      /* optional device pointer (8-byte aligned), read when the kernel runs: a graph
                                  whose caller counts it up draws a new mask with every replay */
} muon_dropout_mask;

/* Arguments of muon_dropout. */
typedef struct muon_dropout_args {
    const void *x;             /* rows x cols, `dtype` */
    const void *add;           /* rows x cols, `dtype`, added after the mask; optional; may be y itself */
    void       *y;             /* rows x cols, `dtype`; may be x itself (same leading dimension) */
    muon_dropout_mask drop;
    int64_t     rows, cols;    /* rows >= 0, 1 <= cols <= 2^20 */
    int64_t     ld_x, ld_add, ld_y;
    int32_t     dtype;
    int32_t     reserved;      /* must be 0 */
} muon_dropout_args;

typedef enum muon_norm {
    MUON_NORM_NONE = 0,
    MUON_NORM_RMS = 1,         /* x / sqrt(sum x^2 / cols + eps) */
    MUON_NORM_LAYER = 2        /* (x - mean) / sqrt(sum (x - mean)^2 / cols + eps) */
} muon_norm;

/* Arguments of muon_blocknorm_forward.  The residual stream (x, s) has
 * `stream_dtype`, the block's own tensors (branch, y) `dtype`; the pair is
 * bf16 and bf16, float32 and float32, or a float32 stream with bf16 blocks. */
typedef struct muon_blocknorm_args {
    const void *x;             /* rows x cols: the stream before the junction */
    const void *branch;        /* rows x cols: the block's output; optional */
    const void *post_gain, *post_bias; /* cols, `param_dtype`: of the branch's norm; optional (bias: layer norm only) */
    const void *gate;          /* cols, `param_dtype`: factors of the branch's columns; optional */
    const void *pre_gain, *pre_bias;   /* of the norm behind the junction; optional (bias: layer norm only) */
    void       *s;             /* rows x cols: the stream behind the junction; may be x (same leading dimension);
                                  NULL without a branch, where x is it */
    void       *y;             /* rows x cols: its norm, the next block's input; NULL with pre_norm NONE */
    muon_act8   y8;            /* y's 8-bit checkpoint, of y before its rounding; codes NULL = none */
    float      *post_mean, *post_rstd, *pre_mean, *pre_rstd;   /* rows; each optional; means: layer norm only */
    muon_dropout_mask drop;    /* of the branch, between its norm and its gate */
    int64_t     rows, cols;    /* rows >= 0, 1 <= cols <= 2^20 */
    int64_t     ld_x, ld_branch, ld_s, ld_y;
    float       residual_scale, branch_scale;   /* finite */
    float       post_eps, pre_eps;     /* >= 0, finite */
    int32_t     post_norm, pre_norm;   /* muon_norm */
    int32_t     stream_dtype, dtype, param_dtype;
    int32_t     reserved;      /* must be 0 */
} muon_blocknorm_args;

/* Arguments of muon_blocknorm_backward. */
typedef struct muon_blocknorm_grad_args {
    const void *dy;            /* rows x cols, `dtype`: gradient at y; NULL with pre_norm NONE */
    const void *ds;            /* rows x cols, `stream_dtype`: gradient at s from behind; optional beside dy */
    const void *s;             /* rows x cols, `stream_dtype`: the stream behind the junction, as stored (x without a
                                  branch); with pre_norm */
    const void *branch;        /* rows x cols, `dtype`; with post_norm, or for dgate */
    const void *post_gain, *post_bias, *gate, *pre_gain;
    const float *post_mean, *post_rstd, *pre_mean, *pre_rstd;  /* as the forward pass wrote them */
    void       *dx;            /* rows x cols, `stream_dtype`; may be ds itself (same leading dimension) */
    void       *dbranch;       /* rows x cols, `dtype`; NULL: the junction had no branch */
    void       *dpost_gain, *dpost_bias, *dgate, *dpre_gain, *dpre_bias;   /* cols, `param_dtype`; each optional */
    muon_dropout_mask drop;
    int64_t     rows, cols;
    int64_t     ld_dy, ld_ds, ld_s, ld_branch, ld_dx, ld_dbranch;
    float       residual_scale, branch_scale;
    int32_t     post_norm, pre_norm;
    int32_t     stream_dtype, dtype, param_dtype;
    int32_t     accumulate;    /* 1: the parameters' gradients are added to */
    int32_t     reserved;      /* must be 0 */
} muon_blocknorm_grad_args;

/* Version of this header the library was built from (MUON_ABI_VERSION). */
int muon_abi_version(void);

/* Create a handle on HIP device `device`.  *out receives the handle (NULL on error).
 * Errors: MUON_ERR_INVALID_ARG (out == NULL, device out of range, unknown flag or role bits),
 * MUON_ERR_NO_DEVICE (no HIP device visible). */
muon_status muon_init(muon_handle **out, int device, uint32_t flags);

/* One Muon step over `n_mats` matrices (all steps above), enqueued on `stream`.
 *
 * Plans.  The first call for a given signature (the list of shapes, blocks,
 * dtypes, update_out presence and compute mode) builds a plan: tile lists,
 * device tables and a workspace of about 7 bytes per weight element in bf16
 * mode plus two min(rows,cols)^2 bf16 squares per matrix, zero-filled, then
 * waits for the stream once.  The handle keeps the plan of every signature it
 * has seen until muon_destroy (grow only): a later call with a known signature
 * allocates nothing and never synchronises, whichever signature came between.
 * Per plan the handle keeps up to 16 device copies of descriptor tables (the
 * call's pointers); a call whose pointers match a resident table enqueues
 * kernel launches only, otherwise it first uploads its table (an
 * asynchronous copy from pinned host memory) over the least recently used one.
 *
 * Graph capture.  A call on a stream that is being captured into a HIP graph
 * must find both its plan and a descriptor table with exactly its pointers
 * resident, i.e. the same call must have run once outside capture; otherwise
 * it returns MUON_ERR_INVALID_ARG and enqueues nothing.  The graph then reads
 * that plan's workspace and that table, which stay allocated and unchanged
 * until muon_destroy (a captured table is never overwritten; later calls with
 * other pointers use other tables).  Replays therefore act on the captured
 * buffers; they share the plan's workspace with eager calls of the same
 * signature, so replays and such calls must be ordered on one stream like any
 * two calls on the handle.  Destroying the handle invalidates the graph.
 *
 * A matrix cut into blocks (block_rows/block_cols) enters the plan as one entry
 * per block, in row-major block order; at most 65536 entries per call.
 * Normalisation is safe at any finite scale: the sum of squares runs in
 * double, and an input whose norm lies outside [2^-30, 2^30] is rescaled by a
 * power of two before the first products (one extra pass over its operand
 * copy; role MUON_ROLE_RESCALE, whose launch returns at once otherwise).
 * n_mats == 0 is a no-op.  Errors: MUON_ERR_INVALID_ARG (null handle/mats/hp with
 * n_mats > 0, null param/grad/momentum, rows or cols < 1, ld < cols, param == grad,
 * momentum aliasing param or grad, ns_steps outside 0..64, a == 0 or a non-finite
 * coefficient, also in coeffs, a block size < 0 or not dividing its dimension,
 * more than 65536 entries, reserved != 0, n_mats < 0, a capturing stream without
 * the resident plan and table described above), MUON_ERR_DTYPE, MUON_ERR_OOM,
 * MUON_ERR_HIP. */
muon_status muon_step(muon_handle *h, const muon_matrix *mats, int32_t n_mats,
                      const muon_hparams *hp, void *stream);

/* muon_step for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation): the
 * same step, with the same arguments, validation, errors and results
 * (bitwise) as muon_step, but every buffer it needs beyond the caller's
 * tensors (workspace, tile lists, units, norm partials, descriptor table)
 * lives in a static device array of 256 MiB per GPU (MUON_STATIC_SCRATCH_BYTES)
 * that the library reserves when it is loaded and holds until the process
 * ends.  Nothing is allocated: no hipMalloc/hipFree, no pinned host memory,
 * no events (profiling handles are not timed here).
 *   - A call whose workspace and tables exceed the scratch returns
 *     MUON_ERR_INVALID_ARG naming both sizes and enqueues nothing (roughly: up
 *     to ~30 M weight elements per call in bf16 mode).
 *   - Every call on a GPU shares that GPU's scratch, which keeps the last
 *     call's contents.  A call whose signature differs from the previous call's
 *     on the device clears the workspace (a fill kernel) and writes its tile
 *     lists; one whose pointers differ writes its descriptor table; either
 *     waits for `stream` before returning (the copies read host memory).  A
 *     call with the previous call's shapes and pointers enqueues kernels only.
 *   - Calls that overlap on one GPU (other streams, other threads, other
 *     handles) race on the scratch: order them.
 *   - The handle is used for its device and error text only; its plans are
 *     neither used nor created. */
#define MUON_STATIC_SCRATCH_BYTES (256u << 20)
muon_status muon_step_noalloc(muon_handle *h, const muon_matrix *mats, int32_t n_mats,
                              const muon_hparams *hp, void *stream);

/* Newton-Schulz only: out = NS(in) for one rows x cols matrix (normalise,
 * transpose rule, hp->ns_steps iterations with hp->a/b/c and hp->eps, in
 * hp->compute precision).  `in` has dtype `in_dtype` and leading dim ld_in;
 * `out` is rows x cols float32 with leading dim ld_out.  beta, lr, weight_decay
 * and nesterov are ignored.  Same errors as muon_step. */
muon_status muon_orthogonalize(muon_handle *h, const void *in, float *out,
                               int64_t rows, int64_t cols, int64_t ld_in, int64_t ld_out,
                               int32_t in_dtype, const muon_hparams *hp, void *stream);

/* One AdamW step over `n` tensors, enqueued on `stream`: for every element
 *
 *   m' = beta1 m + (1 - beta1) g ;  v' = beta2 v + (1 - beta2) g^2
 *   p' = p (1 - lr wd) - lr (m' / (1 - beta1^t)) / (sqrt(v' / (1 - beta2^t)) + eps)
 *
 * in float32 arithmetic (param rounded once to its dtype).  This is the update
 * the hybrid setup runs on the parameters Muon does not take ("14 --
 * modded-nanogpt", section 3; the Muon page, "Where Muon does not apply"); the
 * pages give no formula, so it is the standard AdamW (Loshchilov and Hutter,
 * decoupled weight decay, bias-corrected Adam moments).  One launch covers the
 * whole list.  The first call for a list of sizes/dtypes builds a plan (a few
 * bytes of device tables per 4096 elements); plans and descriptor tables are
 * cached and captured exactly as for muon_step.  n == 0 is a no-op.  Errors: MUON_ERR_INVALID_ARG (null
 * handle/tensors/hp with n > 0, a null buffer with numel > 0, numel < 0,
 * buffers of one tensor aliasing each other, beta outside [0, 1), eps <= 0,
 * a non-finite lr/eps/weight_decay, step < 1, reserved != 0, n < 0, a capturing
 * stream without the resident plan and table), MUON_ERR_DTYPE, MUON_ERR_OOM,
 * MUON_ERR_HIP. */
muon_status muon_adamw_step(muon_handle *h, const muon_adamw_tensor *tensors, int32_t n,
                            const muon_adamw_hparams *hp, void *stream);

/* Layer norm over the rows of x, enqueued on `stream`:
 *
 *   mean = sum x / cols;  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps)
 *   y = (x - mean) rstd gain + bias
 *
 * in float32 (squares past its range make the variance infinite), y rounded
 * once to its dtype.  mean and rstd are kept for the backward pass, y8 holds y
 * for the weight gradient of the layer it feeds.
 *
 * Conventions of the seven layer operators: every matrix is row-major with a
 * leading dimension in elements; any alignment of the element type and any
 * size within the limits named is taken (16-byte aligned rows of whole 16-byte
 * chunks run fastest); rows == 0 enqueues nothing (every matrix with a row per
 * token may then be NULL), except that the gradients of parameters are zeroed
 * (or left, with accumulate).  Nothing but the named outputs is written: a
 * leading dimension's padding keeps its values.  Outputs may not be inputs or
 * each other except where noted (base addresses are compared).
 * Results do not depend on timing: the same call gives the same bits.  They
 * are not among the profiled roles.  Workspaces belong to the handle and grow
 * in blocks of whole MiB, each at least twice the one before (of the size needed
 * where that cannot be had), of which none is freed or moved until muon_destroy,
 * as a graph may use it: doubled blocks together hold less than four times what
 * the largest call needs.  Calls on one handle share them and must be ordered,
 * like those of muon_step (graphs captured from one handle too, when they are
 * replayed).  A call captured into a HIP graph must find its workspace large
 * enough, so a call of the same sizes, leading dimensions and alignments must
 * have run once outside capture (MUON_ERR_INVALID_ARG otherwise).  Errors:
 * MUON_ERR_INVALID_ARG (a null handle, argument struct or required pointer, a
 * size or leading dimension out of range, a product of more than 2^24 - 8 output
 * tiles of 128 x 128, 2^23 rows or more of a norm past 16384 columns, aliasing,
 * an unknown activation or weight layout, both z and z8, act_out without either,
 * an activation without either in muon_linear_grad_input, flags other than 0 and
 * 1, reserved != 0), MUON_ERR_DTYPE, MUON_ERR_NO_DEVICE (the handle's device
 * cannot be selected), MUON_ERR_OOM, MUON_ERR_HIP. */
muon_status muon_layernorm_forward(muon_handle *h, const muon_layernorm_args *args, void *stream);

/* Its gradient: with xh = (x - mean) rstd and a = dy gain,
 *
 *   dx = rstd (a - sum a / cols - xh sum (a xh) / cols) + add
 *   dgain = sum over rows of dy xh;  dbias = sum over rows of dy */
muon_status muon_layernorm_backward(muon_handle *h, const muon_layernorm_grad_args *args, void *stream);

/* y = act(x W + bias) + residual: one matrix product with its epilogue, sums in
 * float32, each output rounded once.  W is in x out (W(i, o) = w[i * ld_w + o])
 * or out x in (w[o * ld_w + i]).  Sums of few rows or few columns are split
 * over workgroups along `in` and joined by a second kernel. */
muon_status muon_linear_forward(muon_handle *h, const muon_linear_args *args, void *stream);

/* dx = (dy W^T) act'(z) + add: the gradient at the pre-activation z of the layer
 * before (act its activation), or at this layer's input without z and z8. */
muon_status muon_linear_grad_input(muon_handle *h, const muon_linear_grad_input_args *args, void *stream);

/* dw = x^T dy (as w is stored), db = the column sums of dy: what muon_step and
 * muon_adamw_step take as gradients. */
muon_status muon_linear_grad_weight(muon_handle *h, const muon_linear_grad_weight_args *args, void *stream);

/* The 8-bit checkpoint `q` of a rows x cols matrix x (dtype, leading dimension
 * ld_x), and back: y = what q stands for, in `dtype`. */
muon_status muon_act_encode(muon_handle *h, const void *x, int64_t rows, int64_t cols, int64_t ld_x,
                            int32_t dtype, const muon_act8 *q, void *stream);
muon_status muon_act_decode(muon_handle *h, const muon_act8 *q, void *y, int64_t rows, int64_t cols,
                            int64_t ld_y, int32_t dtype, void *stream);

/* ---- the block operators ----
 * Conventions, workspaces, capture and errors are those of the seven layer
 * operators (muon_layernorm_forward). */

/* Gated feed-forward: with zg = x Wg + bias_gate and zu = x Wu + bias_up,
 *
 *   h = act(zg) zu
 *
 * both products, the activation and the product in one kernel, sums in float32,
 * h rounded once.  The down projection behind it is muon_linear_forward, its
 * weight's gradient muon_linear_grad_weight. */
muon_status muon_gated_forward(muon_handle *h, const muon_gated_args *args, void *stream);

/* With dh = dy Wd^T, the gradient at h through the down projection,
 *
 *   dgate = dh zu act'(zg),  dup = dh act(zg),  and h = act(zg) zu again */
muon_status muon_gated_grad_hidden(muon_handle *h, const muon_gated_grad_hidden_args *args, void *stream);

/* dx = dgate Wg^T + dup Wu^T + add, one sum */
muon_status muon_gated_grad_input(muon_handle *h, const muon_gated_grad_input_args *args, void *stream);

/* dw_gate = x^T dgate, dw_up = x^T dup (as the weights are stored), db_gate and
 * db_up the column sums of dgate and dup */
muon_status muon_gated_grad_weight(muon_handle *h, const muon_gated_grad_weight_args *args, void *stream);

/* y = x under the mask + add.  The gradient at x is the same call on dy. */
muon_status muon_dropout(muon_handle *h, const muon_dropout_args *args, void *stream);

/* The junction behind a block: with t = norm_post(branch) post_gain + post_bias,
 *
 *   s = residual_scale x + branch_scale gate drop(t)     rounded to the stream's type
 *   y = norm_pre(s) pre_gain + pre_bias                  of s as rounded
 *
 * in one pass over the rows.  Without a branch it is the norm before the first
 * block (residual_scale 1, no post norm, gate or dropout); with pre_norm NONE it
 * ends behind the last one.  An absent gain or gate is 1, an absent bias 0.
 * Squares past float32's range make a row's root infinite. */
muon_status muon_blocknorm_forward(muon_handle *h, const muon_blocknorm_args *args, void *stream);

/* Its gradient: with g = ds + (the gradient of norm_pre at s), e = branch_scale
 * drop(g), and the branch's normalised rows oh (the branch itself without a post norm),
 *
 *   dx = residual_scale g;  dbranch = the gradient of norm_post under e gate post_gain
 *   dpost_gain = sum e gate oh;  dpost_bias = sum e gate;  dgate = sum e t
 *   dpre_gain, dpre_bias: as in muon_layernorm_backward */
muon_status muon_blocknorm_backward(muon_handle *h, const muon_blocknorm_grad_args *args, void *stream);

/* Frobenius norms ||u||_F of the orthogonalised inputs of the most recent
 * muon_step (as enqueued: read after that step's kernels), one per plan entry (a blocked matrix has one per block, row-major)
 * in list order, copied to host memory `out` (n entries; the call
 * synchronises the stream).  Validation hook. */
muon_status muon_read_norms(muon_handle *h, float *out, int32_t n, void *stream);

/* Statistics per kernel role (profiling handles only); returns the number of
 * entries written (<= max), after waiting for the timed launches to finish. */
int32_t muon_kernel_stats_read(muon_handle *h, muon_kernel_stats *out, int32_t max);
void muon_kernel_stats_reset(muon_handle *h);

/* Workspace bytes currently held by the handle: the sum over the plans of
 * every signature seen (the plans' small device tables not included), and the
 * blocks of the layer operators. */
int64_t muon_workspace_bytes(const muon_handle *h);

/* Free the handle and its workspace (waits for the device).  NULL is a no-op. */
muon_status muon_destroy(muon_handle *h);

/* Static text for a status code. */
const char *muon_status_str(muon_status s);

/* Text of the last error on this handle ("" if none); valid until the next call. */
const char *muon_last_error(const muon_handle *h);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_H */

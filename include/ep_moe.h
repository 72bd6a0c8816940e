/*
 * ep_moe.h -- C ABI of the MoE layer's operators of libep_gb300.so: what a
 * user computes around a dispatch and a combine.
 *
 *  - router:  a token's top-k experts and their weights, from its hidden row
 *             (the topk_ids and topk_weights that ep_dispatch takes);
 *  - experts: the experts' products for a few tokens, with bf16 or 4-bit
 *             weights: of all experts (router and experts are then a whole MoE
 *             layer on one GPU) or of one rank's (on the rows a dispatch
 *             delivered, giving the rows a combine adds up);
 *  - linear:  y = x W^T for a few tokens, W in 4 bits with group scales.
 *
 * Statuses, ep_last_error, streams, devices and threads are as in ep.h: every
 * call checks its arguments on the host before it launches anything, queues its
 * work on the given stream and returns. The checked build reports as there, but
 * tests fewer accesses here: the experts' reads of ids and weights, and all
 * stores of ids, weights and results. Reads of x, weights and biases, packed
 * weights and workspaces are not tested.
 * Calls on one handle must be ordered on the device too (one stream, or
 * streams with events between them): a handle's workspace holds one call's
 * intermediate results. Handles are created and destroyed outside stream
 * captures; destroying one waits for its device, so that its workspace can be
 * freed or used again at once. Run calls can be captured. Tensors that a
 * capture or a queued call uses must stay valid until it has run.
 *
 * The blocks of the experts' kernels, and of the router's where it splits the
 * inputs, wait for one another (they are launched cooperatively); every wait,
 * for a copy too, has a limit of about 2 s. If one runs out the kernel ends,
 * that call's output is undefined, and the handle's next call returns
 * EP_ERR_CUDA once.
 */
#ifndef EP_MOE_GB300_H
#define EP_MOE_GB300_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EP_MOE_MAX_TOKENS 64     /* rows of one experts or linear call */
#define EP_MOE_MAX_EXPERTS 512   /* experts of a router; local experts of an experts handle */
#define EP_MOE_MAX_DIM 65536     /* hidden, intermediate, inputs */
#define EP_ROUTER_MAX_TOKENS 2147483136 /* rows of one router call: 2^31 - 512 */

/* ---- router ------------------------------------------------------------------
 * l = x W^T in fp32; s = sigmoid(l), or softmax(l) over the experts.
 * The choice goes by c = s + bias. With num_groups > 1 the experts are split
 * into num_groups equal runs, a group's value is the sum of its two largest
 * c (its largest, for groups of one), and only the top_groups groups with
 * the largest values take part. The top_k experts with the largest c are
 * chosen, in descending order of c. Ties, of groups too, go to the lowest
 * index. A softmax router without bias and groups ranks by l itself.
 * weights = s of the chosen (without bias), divided by their sum if
 * renormalize (scores that are all 0 in fp32 stay 0), times scale.
 * An expert whose c is -infinity (a bias of -infinity masks it) or NaN is
 * never chosen; where fewer than top_k are left, the remaining ids are
 * EP_INVALID_EXPERT_ID with weight 0, which ep_dispatch routes nowhere.
 */
typedef enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 } ep_scoring;

typedef struct ep_router ep_router;

typedef struct {
    int num_experts;    /* 1..EP_MOE_MAX_EXPERTS */
    int top_k;          /* 1..EP_MAX_TOP_K, <= experts in top_groups groups */
    int hidden;         /* a multiple of 8, <= EP_MOE_MAX_DIM */
    ep_dtype dtype;     /* of x and weight: EP_DTYPE_BF16 or EP_DTYPE_FP16 */
    ep_scoring scoring;
    int num_groups;     /* 1, or a divisor of num_experts, <= 32 */
    int top_groups;     /* 1..num_groups */
    int renormalize;    /* 0/1 */
    float scale;        /* finite */
    const void *weight; /* device [num_experts, hidden] of dtype, 16-byte aligned; kept, not copied */
    const float *bias;  /* device [num_experts], or NULL */
} ep_router_config;

ep_status ep_router_create(const ep_router_config *cfg, ep_router **out);

/* Bytes of device workspace a call with num_tokens rows needs (may be 0). */
ep_status ep_router_workspace_size(const ep_router *r, int num_tokens, size_t *bytes);

/* x: device [num_tokens, hidden], rows x_stride elements apart (a multiple
 * of 8, >= hidden), 16-byte aligned; ids: device int32 and weights: device
 * fp32 [num_tokens, top_k], contiguous. workspace: device, 256-byte aligned,
 * of workspace_bytes >= ep_router_workspace_size (used by this call alone).
 * 0 <= num_tokens <= EP_ROUTER_MAX_TOKENS; 0 does nothing. Up to
 * EP_MOE_MAX_TOKENS rows need no workspace. */
ep_status ep_router_run(ep_router *r, const void *x, long long x_stride, int num_tokens, int32_t *ids,
                        float *weights, void *workspace, size_t workspace_bytes, void *stream);

ep_status ep_router_destroy(ep_router *r);

/* ---- 4-bit weights -------------------------------------------------------------
 * w[r][c] = scale[r][c / group] * (code[r][c] - zero[r][c / group])
 * codes 0..15, two to a byte, the even column in the low four bits; zero
 * points 0..15 (8 without them). The operators read them in a packed order:
 * tiles of 128 rows x 128 columns with their scales and zero points.
 */
typedef struct {
    const uint8_t *codes;  /* device [mats, rows, cols / 2] */
    const void *scales;    /* device [mats, rows, cols / group], EP_DTYPE_BF16 or EP_DTYPE_FP16 */
    const uint8_t *zeros;  /* device [mats, rows, cols / group], or NULL */
    ep_dtype scale_dtype;
    int mats, rows, cols;  /* rows, cols >= 1; cols a multiple of group */
    int group;             /* 32, 64 or 128 */
    int gate_up;           /* 0, or 1: matrices are gate and up in turn (mats even), packed for
                              ep_experts_config.gate_up */
} ep_int_weight;

/* A weight as the operators take it: group 0: data is bf16, contiguous,
 * 16-byte aligned, kept and not copied; group 32, 64 or 128: data is what
 * ep_weight_pack wrote. */
typedef struct {
    const void *data;
    int group;
    int has_zeros;         /* packed: with zero points */
    ep_dtype scale_dtype;  /* packed */
} ep_weight;

ep_status ep_weight_packed_size(const ep_int_weight *w, size_t *bytes);

/* Packs w into packed: device, 128-byte aligned, of at least
 * ep_weight_packed_size bytes. w is not needed once the queued work has run.
 * gate_up of experts is packed as 2*experts matrices of `intermediate` rows,
 * with the gate_up field set. The queued work ends with a host function, so
 * that what follows on the stream starts after it in full: ep_linear_run reads
 * its weight before the kernel queued before it has ended. Packed bytes that
 * come from elsewhere are put in place by a copy, not by a kernel right before
 * the call. */
ep_status ep_weight_pack(const ep_int_weight *w, void *packed, size_t bytes, void *stream);

/* ---- linear ----------------------------------------------------------------------
 * y = x W^T with packed 4-bit W [outputs, inputs]: sums are fp32, no weight is
 * rounded, y is rounded once.
 */
typedef struct ep_linear ep_linear;

typedef struct {
    int inputs;       /* a multiple of the group, <= EP_MOE_MAX_DIM */
    int outputs;      /* 1 .. 16 * EP_MOE_MAX_DIM */
    int max_tokens;   /* 1..EP_MOE_MAX_TOKENS */
    ep_weight weight; /* packed, kept */
} ep_linear_config;

ep_status ep_linear_workspace_size(const ep_linear_config *cfg, size_t *bytes);

/* workspace as for ep_experts_create. */
ep_status ep_linear_create(const ep_linear_config *cfg, void *workspace, size_t bytes, ep_linear **out);

/* x: device [num_tokens, inputs], rows x_stride elements apart (a multiple
 * of 8), 16-byte aligned; y: device [num_tokens, outputs], rows y_stride
 * elements apart; both of dtype, EP_DTYPE_BF16 or EP_DTYPE_FP16.
 * 0 <= num_tokens <= max_tokens; 0 does nothing. y may not overlap x. */
ep_status ep_linear_run(ep_linear *h, ep_dtype dtype, const void *x, long long x_stride, int num_tokens, void *y,
                        long long y_stride, void *stream);

ep_status ep_linear_destroy(ep_linear *h);

/* ---- experts -------------------------------------------------------------------
 * y_t = sum_k w_tk * W2_e ( silu(W1_e x_t) * (W3_e x_t) ),  e = ids[t, k] - first_expert
 * over the k whose e lies in [0, num_experts); a token with none gets 0.
 * Sums are fp32, the intermediate row keeps 16 bits of mantissa, y is rounded
 * once to bf16. An id that a token names twice counts twice.
 */
typedef struct ep_experts ep_experts;

typedef struct {
    int num_experts;    /* local experts, 1..EP_MOE_MAX_EXPERTS */
    int first_expert;   /* global id of the first; the last one's fits int32 too */
    int top_k;          /* 1..EP_MAX_TOP_K */
    int hidden;         /* a multiple of 8 (of the group, for 4-bit weights), <= EP_MOE_MAX_DIM */
    int intermediate;   /* likewise */
    int max_tokens;     /* 1..EP_MOE_MAX_TOKENS; after a dispatch: the slots of a receive buffer,
                           ep_size * tokens_per_rank, empty ones included */
    ep_weight gate_up;  /* [num_experts, 2*intermediate, hidden]: gate rows, then up rows */
    ep_weight down;     /* [num_experts, hidden, intermediate] */
} ep_experts_config;

ep_status ep_experts_workspace_size(const ep_experts_config *cfg, size_t *bytes);

/* workspace NULL: allocated with cudaMalloc and freed by ep_experts_destroy;
 * else caller-owned device memory, 256-byte aligned, of at least
 * ep_experts_workspace_size bytes. */
ep_status ep_experts_create(const ep_experts_config *cfg, void *workspace, size_t bytes, ep_experts **out);

/* x, out: device bf16 [num_tokens, hidden], rows x_stride / out_stride
 * elements apart (>= hidden; x_stride a multiple of 8), x 16-byte aligned;
 * ids int32 and weights fp32: device [num_tokens, top_k], contiguous.
 * 0 <= num_tokens <= max_tokens; 0 does nothing. out may not overlap the inputs. */
ep_status ep_experts_run(ep_experts *h, const void *x, long long x_stride, const int32_t *ids,
                         const float *weights, int num_tokens, void *out, long long out_stride, void *stream);

ep_status ep_experts_destroy(ep_experts *h);

/* A whole MoE layer: ep_router_run, then ep_experts_run on its ids and
 * weights (which are outputs here). Both handles have the same hidden size
 * and top_k, the router's dtype is bf16; num_tokens <= max_tokens. */
ep_status ep_layer_run(ep_router *r, ep_experts *h, const void *x, long long x_stride, int num_tokens,
                       int32_t *ids, float *weights, void *out, long long out_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_MOE_GB300_H */

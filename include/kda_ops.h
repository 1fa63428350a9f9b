/*
 * kda_ops.h -- the operators a serving decoder runs around Kimi Delta Attention
 * (kda.h): the short causal convolution in front of a KDA layer, the query /
 * key norm with the position rotation in front of a softmax-attention layer,
 * and the attention that verifies drafted tokens (a tree, a chain, or one
 * token) over that layer's paged cache.
 *
 * Conventions are those of kda.h: device pointers owned by the caller, element
 * strides, asynchronous calls on `stream`, host errors returned synchronously
 * with nothing launched, device-only errors written to *device_status (when
 * non-NULL) while the kernels skip the offending work, 16-byte aligned base
 * pointers and strides that are multiples of 8 elements (KDA_ERR_UNSUPPORTED
 * otherwise).  No call allocates memory.
 */
#ifndef KDA_OPS_H
#define KDA_OPS_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define KDA_DTYPE_BF16 0
#define KDA_DTYPE_F16 1
#define KDA_DTYPE_F32 2

/*
 * Short causal convolution of a KDA layer's projections (depthwise: channel c
 * sees only channel c), its activation, and the per-head L2 norm of the q and k
 * channels.  For a sequence with tokens x_0 .. x_{L-1} and the W - 1 inputs
 * before them x_{-(W-1)} .. x_{-1}:
 *
 *     z_t[c] = bias[c] + sum_{j < W} weight[c][j] x_{t-W+1+j}[c]
 *     y_t[c] = z / (1 + e^{-z})                (silu = 1)  or  z  (silu = 0)
 *     y_t[c] /= sqrt(sum over its head of 128 channels of y_t^2 + norm_eps)
 *                                              (channels c < norm_channels)
 *
 * in fp32, rounded once to the element type of x.  (With silu z has to be below
 * 2^127; under the root fp32 numbers below 2^-126 count as 0, which only a norm_eps
 * below that leaves to be seen.)
 *
 * Sequences: padded (cu_seqlens NULL): num_seqs sequences of seqlen tokens,
 * element (n, t, c) of x at n*x_stride[0] + t*x_stride[1] + c; packed: device
 * int32 cu_seqlens [num_seqs + 1] over seqlen tokens in all, stride [0] unused.
 * One token per sequence is the decoding form, a few the drafts of kda_verify.
 *
 * conv_state (may be NULL: zeros before every sequence, nothing kept): element
 * type of x, [pool_size, W - 1, C] contiguous, row i the i-th oldest input.
 * Sequence n uses entry slot[n] (slot NULL: n); slots must be distinct.
 * has_state (device int32 [num_seqs], NULL: all 1): where 0, the sequence
 * starts from zeros and the entry's old content is not used.  Afterwards the
 * entry holds the last W - 1 inputs up to and including the sequence's first
 * accepted[n] tokens (device int32 [num_seqs], 0 .. length; NULL: all tokens).
 * out == NULL: only the states are updated (the commit of accepted drafts).
 * A slot or accepted entry out of range is reported in device_status and the
 * sequence is left out.  cu_seqlens that does not run from 0 to seqlen without
 * decreasing is reported too, and which of the call's sequences are computed is
 * then not defined (rows of x and out and pool entries of the call alone are used).
 *
 * C (channels) a multiple of 8, W in 2..4, norm_channels a multiple of 128 of
 * at most C; x and out do not overlap.  weight [C, W] and bias [C] contiguous.
 * Size limits: fewer than 2^31 tokens, at most 2^24 channels, num_seqs <= 2^30.
 */
typedef struct kda_short_conv_args {
    const void* x;
    void* out;                  /* element type of x; or NULL */
    const void* weight;         /* [C, W], weight_dtype */
    const float* bias;          /* fp32 [C] or NULL */
    void* conv_state;           /* [pool_size, W - 1, C] or NULL */
    const int32_t* slot;
    const int32_t* has_state;
    const int32_t* accepted;
    const int32_t* cu_seqlens;
    int32_t* device_status;
    int64_t x_stride[2];        /* (sequence, token) element strides */
    int64_t out_stride[2];
    int64_t num_seqs;
    int64_t seqlen;             /* padded: tokens a sequence; packed: tokens in all */
    int64_t channels;
    int64_t norm_channels;
    int64_t pool_size;
    int32_t width;              /* W */
    int32_t dtype;              /* KDA_DTYPE_BF16 or KDA_DTYPE_F16 */
    int32_t weight_dtype;       /* dtype or KDA_DTYPE_F32 */
    int32_t silu;
    float norm_eps;
} kda_short_conv_args;
kda_status kda_short_conv(const kda_short_conv_args* args, void* stream);

/*
 * RMS norm of every query and key head and the rotation by the token's
 * position, in one pass over q and k:
 *
 *     y = x / sqrt(mean(x^2) + norm_eps) * weight   (norm = 1; else y = x, the weights unread)
 *     (a, b) -> s (a cos t - b sin t, a sin t + b cos t),   t = position * inv_freq[i],
 *
 * for i < rot_dim / 2, s = rope_scale, on the pairs (a, b) = (y[i], y[i + rot_dim/2])
 * or, with interleaved = 1, (y[2i], y[2i+1]); channels from rot_dim on keep y.
 * (The root as in kda_short_conv.)
 * Long contexts are a matter of inv_freq and rope_scale.  The angle is formed
 * and reduced with an error below 1e-6 turns for every int32 position and
 * frequencies up to 2^20.
 *
 * q element (b, t, h, c) at b*s[0] + t*s[1] + h*s[2] + c, likewise k, v and the
 * outputs; positions (and slots) at b*seqlen + t, contiguous.  q_out / k_out
 * may be q / k themselves (same pointer and strides), otherwise no overlap.
 *
 * With slots (device int64): key row (b, t) also goes to the cache row slots[b, t]
 * = page * page_size + offset, element h*stride[2] + c of
 * page*stride[0] + offset*stride[1], and v (unchanged) to the same row of
 * v_cache; k_out may then be NULL.  A negative slot writes no cache row; one
 * past the cache is reported in device_status and skipped.
 *
 * head_dim a multiple of 16, at most 256; rot_dim 0 or a multiple of 16, at
 * most head_dim; weights contiguous [head_dim], NULL = ones.  Size limit: fewer
 * than 2^31 tokens, at most 65535 heads.
 */
typedef struct kda_qk_norm_rope_args {
    const void* q;
    const void* k;
    const void* v;              /* NULL unless v_cache */
    void* q_out;
    void* k_out;                /* NULL only with k_cache */
    void* k_cache;
    void* v_cache;              /* NULL: only keys are cached */
    const int64_t* slots;
    const int32_t* positions;
    const float* inv_freq;      /* fp32 [rot_dim / 2] */
    const void* q_weight;
    const void* k_weight;
    int32_t* device_status;
    int64_t q_stride[3];        /* (batch, token, head) element strides */
    int64_t k_stride[3];
    int64_t v_stride[3];
    int64_t q_out_stride[3];
    int64_t k_out_stride[3];
    int64_t k_cache_stride[3];  /* (page, token, head) element strides */
    int64_t v_cache_stride[3];
    int64_t batch;
    int64_t seqlen;
    int64_t num_q_heads;
    int64_t num_k_heads;
    int64_t head_dim;
    int64_t rot_dim;
    int64_t num_pages;
    int64_t page_size;
    int32_t dtype;              /* KDA_DTYPE_BF16 or KDA_DTYPE_F16 */
    int32_t weight_dtype;       /* dtype or KDA_DTYPE_F32 */
    int32_t norm;
    int32_t interleaved;
    float norm_eps;
    float rope_scale;
} kda_qk_norm_rope_args;
kda_status kda_qk_norm_rope(const kda_qk_norm_rope_args* args, void* stream);

/*
 * Attention of drafted tokens over a paged cache.  Request r has a context of
 * context_lens[r] tokens and num_nodes[r] <= max_nodes drafted tokens (NULL: all
 * max_nodes), whose keys and values are in the cache behind the context's:
 * position p < context_lens[r] + num_nodes[r] is row p mod page_size of page
 * page_table[r][p / page_size].  Node i of r sees every context token, and node
 * j where bit j mod 64 of tree_mask[r][i][j / 64] is set (tree_mask NULL: the
 * nodes j <= i, a chain; a single token is max_nodes = 1).  With S_i the set of
 * positions that node i sees, query head h and key head h / (Hq / Hk):
 *
 *     out_i = sum_{p in S_i} e^{scale q_i.k_p - m} v_p / sum_{p in S_i} e^{scale q_i.k_p - m},
 *     lse_i = ln sum_{p in S_i} e^{scale q_i.k_p}
 *
 * An empty S_i (and every row past num_nodes[r]) gives out = 0 and lse = -inf.
 * Keys and values that a node does not see have no influence on it, whatever
 * they hold (NaN and infinities too).  Products and sums are fp32; the weights
 * e^{..} enter the product with v in the element type (fp16: scaled, so that those
 * down to 2^-35 of the largest are kept).
 *
 * q and out element (r, i, h, c) at r*s[0] + i*s[1] + h*s[2] + c; cache element
 * (page, row, h, c) likewise; tree_mask contiguous [R, max_nodes, ceil(max_nodes/64)];
 * lse contiguous fp32 [R, max_nodes, Hq] or NULL; page_table row r at
 * r*page_table_stride.  out may be q itself (same pointer and strides; head size
 * 256 then takes the kernel for few rows whatever their number), otherwise no
 * overlap.
 * head_dim 64, 128 or 256; Hq a multiple of Hk; max_nodes <= 256.
 * max_context: an upper bound of context_lens that the host knows (<= 0: what
 * the page table can address); it sets how the work is cut, not the result's
 * definition.  Give it where the table is much wider than the contexts: 4 requests
 * of 5 drafts and 4 query heads a key head over up to 1000 tokens, in a table for
 * 131072, take 10.7 us with it and 17.8 without, one token over 1000 tokens 7.5
 * and 9.5.  A context length or node count out of range gives the request
 * zero rows; a page outside 0 .. num_pages - 1 reads as zeros; both are
 * reported in device_status.
 * workspace: kda_tree_attention_workspace_size(args) bytes, 256-byte aligned,
 * used during the call's kernels only.
 * Size limits: R <= 65535, Hk <= 65535, contexts below 2^30 tokens.
 */
typedef struct kda_tree_attention_args {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    void* out;
    float* lse;
    const int32_t* page_table;
    const int32_t* context_lens;
    const int32_t* num_nodes;
    const uint64_t* tree_mask;
    void* workspace;
    int32_t* device_status;
    size_t workspace_bytes;
    int64_t q_stride[3];        /* (request, node, head) element strides */
    int64_t out_stride[3];
    int64_t k_cache_stride[3];  /* (page, row, head) element strides */
    int64_t v_cache_stride[3];
    int64_t page_table_stride;
    int64_t num_requests;
    int64_t max_nodes;
    int64_t num_q_heads;
    int64_t num_k_heads;
    int64_t head_dim;
    int64_t num_pages;
    int64_t page_size;
    int64_t pages_per_request;  /* columns of page_table */
    int64_t max_context;
    int32_t dtype;              /* KDA_DTYPE_BF16 or KDA_DTYPE_F16 */
    float scale;
} kda_tree_attention_args;
size_t kda_tree_attention_workspace_size(const kda_tree_attention_args* args);
kda_status kda_tree_attention(const kda_tree_attention_args* args, void* stream);
/*
 * The same with overrides for tests (NULL: none): wait_limit_ns and timeout_probe
 * apply to the kernel for many rows, whose waits are the only ones of these
 * operators: bounded by wait_limit_ns (200 ms by default) and 0.1 ms for every 128
 * tokens of the longest context, since some last as long as a context's work.  A
 * wait that runs out reports KDA_ERR_TIMEOUT in device_status.
 */
kda_status kda_tree_attention_ex(const kda_tree_attention_args* args, const kda_overrides* overrides, void* stream);
/*
 * How kda_tree_attention cuts these arguments on a GPU with num_sms SMs (host only:
 * no device call, pointers are not followed).  kernel: KDA_TREE_ITEMS, one CTA a
 * (request, key head, block of rows), the requests longest first where ordered is 1;
 * KDA_TREE_CLUSTERS, `cluster` CTAs each; KDA_TREE_LINE, equal stretches of all of
 * them in a row; KDA_TREE_MANY_ROWS, the kernel for many rows in `launches` launches
 * of up to 256 requests (a cache without a tensor map and results over queries of
 * head size 256 take KDA_TREE_ITEMS or _LINE all the same).  KDA_ERR_INVALID_ARG for
 * NULL or num_sms < 1, otherwise what kda_tree_attention would refuse.
 */
#define KDA_TREE_ITEMS 0
#define KDA_TREE_CLUSTERS 1
#define KDA_TREE_LINE 2
#define KDA_TREE_MANY_ROWS 3
typedef struct kda_tree_schedule {
    int32_t kernel, ordered, cluster, launches;
} kda_tree_schedule;
kda_status kda_tree_attention_schedule(const kda_tree_attention_args* args, int num_sms, kda_tree_schedule* schedule);

#ifdef __cplusplus
}
#endif
#endif /* KDA_OPS_H */

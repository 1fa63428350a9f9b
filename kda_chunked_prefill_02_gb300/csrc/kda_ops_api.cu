// kda_ops_api.cu -- the C ABI of include/kda_ops.h: host-side argument checks
// and the launches.  Nothing here allocates or caches device memory.
#include <math.h>
#include <string.h>

#include "../../include/kda_ops.h"
#include "kda_internal.h"
#include "ops_internal.h"
#include "sm103.cuh"

using namespace kda;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <int N>
bool strides8(const int64_t (&s)[N]) {
    for (int i = 0; i < N; ++i)
        if (s[i] < 0 || s[i] % 8) return false;
    return true;
}
// Results at their inputs' address lie over them row by row (dims of size 1 aside).
template <int N>
bool in_place_or_apart(const void* in, const int64_t (&is)[N], const void* out, const int64_t (&os)[N],
                       const int64_t (&sizes)[N]) {
    for (int i = 0; i < N; ++i)
        if (in == out && sizes[i] > 1 && is[i] != os[i]) return false;
    return true;
}
bool elem_type(int32_t t) { return t == KDA_DTYPE_BF16 || t == KDA_DTYPE_F16; }
kda_status status_of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

kda_status check_tree(const kda_tree_attention_args* a) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->num_requests < 0 || a->max_nodes < 1 || a->num_q_heads < 1 || a->num_k_heads < 1 || a->num_pages < 0 ||
        a->page_size < 1 || a->pages_per_request < 0 || a->num_q_heads % a->num_k_heads != 0 || !isfinite(a->scale))
        return KDA_ERR_INVALID_ARG;
    if (!elem_type(a->dtype) || (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256) ||
        a->max_nodes > 256 || a->num_requests > 65535 || a->num_k_heads > 65535 ||
        a->num_q_heads / a->num_k_heads > 65536 || a->num_pages > INT32_MAX || a->page_size > (1 << 30) ||
        a->pages_per_request > INT32_MAX || a->page_table_stride < 0)
        return KDA_ERR_UNSUPPORTED;
    if (a->num_requests == 0) return KDA_OK;
    if (!a->q || !a->k_cache || !a->v_cache || !a->out || !a->page_table || !a->context_lens || a->num_pages < 1)
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(a->q) || !aligned16(a->k_cache) || !aligned16(a->v_cache) || !aligned16(a->out) ||
        !strides8(a->q_stride) || !strides8(a->out_stride) || !strides8(a->k_cache_stride) ||
        !strides8(a->v_cache_stride))
        return KDA_ERR_UNSUPPORTED;
    const int64_t sizes[3] = {a->num_requests, a->max_nodes, a->num_q_heads};
    if (!in_place_or_apart(a->q, a->q_stride, a->out, a->out_stride, sizes)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Tokens of the longest request the call allows for, or -1 past 2^30.
int64_t tree_max_len(const kda_tree_attention_args* a) {
    const int64_t room = a->pages_per_request * a->page_size;
    int64_t len = room;
    if (a->max_context > 0 && a->max_context < room - a->max_nodes) len = a->max_context + a->max_nodes;
    return len > (1 << 30) ? -1 : len;
}

int sm_count_or_default() {
    const int n = device_sm_count();
    return n > 0 ? n : 152;   // no device (a host-only query of the workspace)
}

TreePlan plan_of(const kda_tree_attention_args* a, int64_t max_len, int num_sms) {
    return tree_plan((int)a->num_requests, (int)a->num_k_heads,
                     (int)(a->max_nodes * (a->num_q_heads / a->num_k_heads)), (int)a->head_dim, max_len,
                     (int)a->page_size, a->scale, num_sms);
}

size_t tree_workspace(const kda_tree_attention_args* a, const TreePlan& plan) {
    return plan.parts * sizeof(int4) + plan.part_rows * ((size_t)a->head_dim + 1) * sizeof(float) +
           plan.order * sizeof(int32_t);
}

}  // namespace

extern "C" {

kda_status kda_short_conv(const kda_short_conv_args* a, void* stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->seqlen < 0 || a->channels < 1 || a->norm_channels < 0 ||
        a->norm_channels > a->channels || a->pool_size < 0 || !(a->norm_eps >= 0.f))
        return KDA_ERR_INVALID_ARG;
    if (a->width < 2 || a->width > 4 || a->channels % 8 || a->norm_channels % kHeadDim || !elem_type(a->dtype) ||
        (a->weight_dtype != a->dtype && a->weight_dtype != KDA_DTYPE_F32) || a->channels > (1 << 24) ||
        a->num_seqs > (1 << 30) || a->pool_size > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    if (a->num_seqs == 0) return a->cu_seqlens && a->seqlen > 0 ? KDA_ERR_INVALID_ARG : KDA_OK;
    if (a->seqlen > INT32_MAX || (!a->cu_seqlens && a->seqlen * a->num_seqs > INT32_MAX)) return KDA_ERR_UNSUPPORTED;
    const int64_t total = a->cu_seqlens ? a->seqlen : a->seqlen * a->num_seqs;
    if (!a->weight || (total > 0 && !a->x) || (!a->out && !a->conv_state) ||
        (a->conv_state && a->pool_size < 1) || (total > 0 && a->out == a->x))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(a->x) || !aligned16(a->out) || !aligned16(a->conv_state) ||
        !aligned16(a->weight) || !aligned16(a->bias) || !strides8(a->x_stride) ||
        (a->out && !strides8(a->out_stride)))
        return KDA_ERR_UNSUPPORTED;
    const int sms = device_sm_count();
    if (sms < 1) return KDA_ERR_CUDA;
    ConvParams p;
    memset(&p, 0, sizeof(p));
    p.x = a->x; p.out = a->out; p.w = a->weight; p.bias = a->bias; p.pool = a->conv_state;
    p.slot = a->slot; p.has_state = a->has_state; p.accepted = a->accepted; p.cu = a->cu_seqlens;
    p.status = a->device_status;
    for (int i = 0; i < 2; ++i) { p.xs[i] = a->x_stride[i]; p.os[i] = a->out_stride[i]; }
    p.N = (int)a->num_seqs; p.T = (int)a->seqlen; p.total = total;
    p.C = (int)a->channels; p.norm_c = (int)a->norm_channels; p.P = (int)a->pool_size;
    p.silu = a->silu ? 1 : 0; p.eps = a->norm_eps;
    return status_of(launch_short_conv(p, a->width, a->dtype == KDA_DTYPE_F16, a->weight_dtype == KDA_DTYPE_F32, sms,
                                       static_cast<cudaStream_t>(stream)));
}

kda_status kda_qk_norm_rope(const kda_qk_norm_rope_args* a, void* stream) {
    if (!a) return KDA_ERR_INVALID_ARG;
    if (a->batch < 0 || a->seqlen < 0 || a->num_q_heads < 0 || a->num_k_heads < 0 ||
        a->num_q_heads + a->num_k_heads < 1 || a->head_dim < 1 || a->rot_dim < 0 || a->rot_dim > a->head_dim ||
        !(a->norm_eps >= 0.f) || !isfinite(a->rope_scale))
        return KDA_ERR_INVALID_ARG;
    if (!elem_type(a->dtype) || (a->weight_dtype != a->dtype && a->weight_dtype != KDA_DTYPE_F32) ||
        a->head_dim % 16 || a->head_dim > 256 || a->rot_dim % 16 || a->num_q_heads > 65535 ||
        a->num_k_heads > 65535 || a->batch > INT32_MAX || a->seqlen > INT32_MAX ||
        a->batch * a->seqlen > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    const int64_t tokens = a->batch * a->seqlen;
    if (tokens == 0) return KDA_OK;
    const bool cached = a->k_cache != nullptr;
    if ((a->num_q_heads > 0 && (!a->q || !a->q_out)) || (a->num_k_heads > 0 && (!a->k || (!a->k_out && !cached))) ||
        (a->rot_dim > 0 && (!a->positions || !a->inv_freq)) || (cached != (a->slots != nullptr)) ||
        (a->v_cache && (!cached || !a->v)) || (cached && (a->page_size < 1 || a->num_pages < 1)))
        return KDA_ERR_INVALID_ARG;
    if (cached && (a->page_size > INT32_MAX || a->num_pages > INT32_MAX)) return KDA_ERR_UNSUPPORTED;
    const void* ptrs[] = {a->q, a->k, a->v, a->q_out, a->k_out, a->k_cache, a->v_cache,
                          a->q_weight, a->k_weight};
    for (const void* ptr : ptrs)
        if (!aligned16(ptr)) return KDA_ERR_UNSUPPORTED;
    if ((a->num_q_heads > 0 && (!strides8(a->q_stride) || !strides8(a->q_out_stride))) ||
        (a->num_k_heads > 0 && (!strides8(a->k_stride) || (a->k_out && !strides8(a->k_out_stride)))) ||
        (cached && !strides8(a->k_cache_stride)) ||
        (a->v_cache && (!strides8(a->v_stride) || !strides8(a->v_cache_stride))))
        return KDA_ERR_UNSUPPORTED;
    const int64_t q_sizes[3] = {a->batch, a->seqlen, a->num_q_heads}, k_sizes[3] = {a->batch, a->seqlen, a->num_k_heads};
    if ((a->num_q_heads > 0 && !in_place_or_apart(a->q, a->q_stride, a->q_out, a->q_out_stride, q_sizes)) ||
        (a->num_k_heads > 0 && a->k_out && !in_place_or_apart(a->k, a->k_stride, a->k_out, a->k_out_stride, k_sizes)))
        return KDA_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms < 1) return KDA_ERR_CUDA;
    RopeParams p;
    memset(&p, 0, sizeof(p));
    p.q = a->q; p.k = a->k; p.v = a->v; p.q_out = a->q_out; p.k_out = a->k_out;
    p.k_cache = a->k_cache; p.v_cache = a->v_cache; p.slots = a->slots; p.positions = a->positions;
    p.inv_freq = a->inv_freq; p.status = a->device_status;
    if (a->norm) { p.q_w = a->q_weight; p.k_w = a->k_weight; }   // the weights are the norm's
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = a->q_stride[i]; p.ks[i] = a->k_stride[i]; p.vs[i] = a->v_stride[i];
        p.qos[i] = a->q_out_stride[i]; p.kos[i] = a->k_out_stride[i];
        p.kcs[i] = a->k_cache_stride[i]; p.vcs[i] = a->v_cache_stride[i];
    }
    p.tokens = tokens; p.T = (int)a->seqlen;
    p.Hq = (int)a->num_q_heads; p.Hk = (int)a->num_k_heads; p.D = (int)a->head_dim; p.rot = (int)a->rot_dim;
    p.cache_rows = cached ? a->num_pages * a->page_size : 0;
    p.page = cached ? (int)a->page_size : 1;
    p.norm = a->norm ? 1 : 0; p.interleaved = a->interleaved ? 1 : 0;
    p.w_f32 = a->weight_dtype == KDA_DTYPE_F32 ? 1 : 0;
    p.eps = a->norm_eps; p.scale = a->rope_scale;
    return status_of(launch_qk_norm_rope(p, a->dtype == KDA_DTYPE_F16, sms, static_cast<cudaStream_t>(stream)));
}

size_t kda_tree_attention_workspace_size(const kda_tree_attention_args* a) {
    if (check_tree(a) != KDA_OK || a->num_requests == 0) return 0;
    const int64_t max_len = tree_max_len(a);
    return max_len < 0 ? 0 : tree_workspace(a, plan_of(a, max_len, sm_count_or_default()));
}

kda_status kda_tree_attention_schedule(const kda_tree_attention_args* a, int num_sms, kda_tree_schedule* schedule) {
    if (!schedule || num_sms < 1) return KDA_ERR_INVALID_ARG;
    memset(schedule, 0, sizeof(*schedule));
    const kda_status st = check_tree(a);
    if (st != KDA_OK || a->num_requests == 0) return st;
    const int64_t max_len = tree_max_len(a);
    if (max_len < 0) return KDA_ERR_UNSUPPORTED;
    const TreePlan plan = plan_of(a, max_len, num_sms);
    schedule->kernel = plan.mma ? KDA_TREE_MANY_ROWS
                                : plan.line ? KDA_TREE_LINE : plan.cluster > 1 ? KDA_TREE_CLUSTERS : KDA_TREE_ITEMS;
    schedule->ordered = plan.order > 0 ? 1 : 0;
    schedule->cluster = plan.mma ? 1 : plan.cluster;
    schedule->launches = plan.mma ? (int)((a->num_requests + kTreeSlice - 1) / kTreeSlice) : 1;
    return KDA_OK;
}

kda_status kda_tree_attention(const kda_tree_attention_args* a, void* stream) {
    return kda_tree_attention_ex(a, nullptr, stream);
}

kda_status kda_tree_attention_ex(const kda_tree_attention_args* a, const kda_overrides* overrides, void* stream) {
    const kda_status st = check_tree(a);
    if (st != KDA_OK || a->num_requests == 0) return st;
    const int64_t max_len = tree_max_len(a);
    if (max_len < 0) return KDA_ERR_UNSUPPORTED;
    if (device_sm_count() < 1) return KDA_ERR_CUDA;
    const TreePlan plan = plan_of(a, max_len, sm_count_or_default());
    const size_t need = tree_workspace(a, plan);
    if (need && (!a->workspace || a->workspace_bytes < need)) return KDA_ERR_INVALID_ARG;
    if (need && (reinterpret_cast<uintptr_t>(a->workspace) & 255u)) return KDA_ERR_UNSUPPORTED;
    TreeParams p;
    memset(&p, 0, sizeof(p));
    p.q = a->q; p.kc = a->k_cache; p.vc = a->v_cache; p.out = a->out; p.lse = a->lse;
    p.table = a->page_table; p.ctx = a->context_lens; p.nodes = a->num_nodes; p.mask = a->tree_mask;
    p.status = a->device_status;
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = a->q_stride[i]; p.os[i] = a->out_stride[i];
        p.ks[i] = a->k_cache_stride[i]; p.vs[i] = a->v_cache_stride[i];
    }
    p.table_stride = a->page_table_stride;
    p.R = (int)a->num_requests; p.N = (int)a->max_nodes; p.Hq = (int)a->num_q_heads; p.Hk = (int)a->num_k_heads;
    p.G = p.Hq / p.Hk; p.rows = p.N * p.G; p.words = (p.N + 63) / 64;
    p.P = (int)a->num_pages; p.page = (int)a->page_size; p.max_len = max_len;
    auto magic = [](int d) { return d == 1 ? 0xffffffffu : (uint32_t)((1ull << 32) / (uint32_t)d); };
    p.page_magic = magic(p.page);
    p.group_magic = magic(p.G);
    p.cluster = plan.cluster;
    p.parts = static_cast<int4*>(a->workspace);
    p.part_o = reinterpret_cast<float*>(p.parts + plan.parts);
    p.part_lse = p.part_o + plan.part_rows * a->head_dim;
    p.order = plan.order ? reinterpret_cast<int32_t*>(p.part_lse + plan.part_rows) : nullptr;
    p.scale_log2 = a->scale * 1.4426950408889634f;
    p.wait_ns = overrides && overrides->wait_limit_ns > 0 ? (uint64_t)overrides->wait_limit_ns : kWaitLimitNs;
    p.timeout_probe = overrides && overrides->timeout_probe ? 1 : 0;
    return status_of(launch_tree_attention(p, plan, (int)a->head_dim, a->dtype == KDA_DTYPE_F16,
                                           static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

"""ctypes binding of the operators in include/kda_ops.h: argument marshalling only.

The operators a serving decoder runs around KDA: the short causal convolution
(`kda_short_conv`), the query / key norm with the position rotation
(`kda_qk_norm_rope`, frequencies from `rope_frequencies`), and the attention of
drafted tokens over a paged cache (`kda_tree_attention`, masks from
`tree_mask`).  As in kda.py, outputs and workspaces come from torch, any status
other than KDA_OK raises KdaError, and there is no fallback.
"""
import ctypes
import math

import torch

from .kda import KdaError, _need_cuda, _on_stream, _stream_handle, lib

KDA_DTYPE_BF16, KDA_DTYPE_F16, KDA_DTYPE_F32 = range(3)
_DTYPES = {torch.bfloat16: KDA_DTYPE_BF16, torch.float16: KDA_DTYPE_F16}

_p, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


def _fields(spec):
    """ctypes fields from "type: name name ..." lines; name[n] is n fields."""
    kinds = {"p": _p, "i64": _i64, "i32": _i32, "f32": _f32, "size": ctypes.c_size_t}
    out = []
    for line in spec.strip().splitlines():
        kind, names = line.split(":")
        for name in names.split():
            base, _, n = name.partition("[")
            count = int(n[:-1]) if n else 0
            out += [("%s%d" % (base, i), kinds[kind.strip()]) for i in range(count)] if n else \
                [(base, kinds[kind.strip()])]
    return out


class ShortConvArgs(ctypes.Structure):
    _fields_ = _fields("""
        p: x out weight bias conv_state slot has_state accepted cu_seqlens device_status
        i64: x_stride[2] out_stride[2] num_seqs seqlen channels norm_channels pool_size
        i32: width dtype weight_dtype silu
        f32: norm_eps""")


class QkNormRopeArgs(ctypes.Structure):
    _fields_ = _fields("""
        p: q k v q_out k_out k_cache v_cache slots positions inv_freq q_weight k_weight device_status
        i64: q_stride[3] k_stride[3] v_stride[3] q_out_stride[3] k_out_stride[3] k_cache_stride[3] v_cache_stride[3]
        i64: batch seqlen num_q_heads num_k_heads head_dim rot_dim num_pages page_size
        i32: dtype weight_dtype norm interleaved
        f32: norm_eps rope_scale""")


class TreeAttentionArgs(ctypes.Structure):
    _fields_ = _fields("""
        p: q k_cache v_cache out lse page_table context_lens num_nodes tree_mask workspace device_status
        size: workspace_bytes
        i64: q_stride[3] out_stride[3] k_cache_stride[3] v_cache_stride[3] page_table_stride
        i64: num_requests max_nodes num_q_heads num_k_heads head_dim num_pages page_size pages_per_request max_context
        i32: dtype
        f32: scale""")


_funcs = None


def _fn():
    global _funcs
    if _funcs is None:
        L = lib()
        for name, args in (("kda_short_conv", ShortConvArgs), ("kda_qk_norm_rope", QkNormRopeArgs),
                           ("kda_tree_attention", TreeAttentionArgs)):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.POINTER(args), _p]
        L.kda_tree_attention_workspace_size.restype = ctypes.c_size_t
        L.kda_tree_attention_workspace_size.argtypes = [ctypes.POINTER(TreeAttentionArgs)]
        _funcs = L
    return _funcs


def _addr(t):
    return None if t is None else t.data_ptr()


def _elem(name, t):
    """KDA_DTYPE_* of a bf16 or fp16 CUDA tensor."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be bf16 or fp16, got %s" % (name, t.dtype))
    return code


def _flat(name, t, dtype, shape):
    """Checks an optional contiguous CUDA tensor of one type and shape."""
    if t is None:
        return
    _need_cuda(name, t, dtype)
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous of shape %s, got %s" % (name, shape, tuple(t.shape)))


def _weight(name, t, dtype, shape):
    """The same for a weight in fp32 or the data's type; returns its KDA_DTYPE_*."""
    if t is None:
        return KDA_DTYPE_F32
    _flat(name, t, torch.float32 if t.dtype == torch.float32 else dtype, shape)
    return KDA_DTYPE_F32 if t.dtype == torch.float32 else _DTYPES[dtype]


def _status(t):
    if t is not None:
        _need_cuda("device_status", t, torch.int32)


def kda_short_conv(x, weight, *, bias=None, conv_state=None, slot=None, has_state=None, cu_seqlens=None,
                   accepted=None, silu=True, norm_channels=0, norm_eps=1e-6, out=None, state_only=False,
                   device_status=None, stream=None):
    """Short causal convolution of a KDA layer (see kda_short_conv in
    include/kda_ops.h); conv_state is updated in place.

    x bf16 or fp16 [B, T, C], or [T_total, C] with cu_seqlens (int32 [N+1] on the
    device); weight [C, W] in x's type or fp32; bias fp32 [C]; conv_state
    [P, W-1, C] in x's type, entry slot[n] (int32 [N], default n) belongs to
    sequence n and holds its last W-1 inputs; has_state int32 [N]: 0 starts the
    sequence from zeros; accepted int32 [N]: the state kept is that after the
    sequence's first accepted[n] tokens.  The first norm_channels channels are
    L2-normalised per head of 128.  Returns out; with state_only=True only the
    states are updated (returns None).
    """
    dtype = _elem("x", x)
    shape, xs = x.shape, x.stride()
    if len(shape) != (2 if cu_seqlens is not None else 3):
        raise ValueError("x must be [T_total, C] with cu_seqlens, [B, T, C] without")
    if xs[-1] != 1:
        raise ValueError("the channel (last) dim must have stride 1")
    C = shape[-1]
    if cu_seqlens is not None:
        _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
        if cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must be contiguous int32 [N+1]")
        N, T, x_stride = cu_seqlens.shape[0] - 1, shape[0], (0, xs[0])
    else:
        N, T, x_stride = shape[0], shape[1], (xs[0], xs[1])
    if weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    weight_dtype = _weight("weight", weight, x.dtype, (C, W))
    _flat("bias", bias, torch.float32, (C,))
    P = 0
    if conv_state is not None:
        P = conv_state.shape[0]
        _flat("conv_state", conv_state, x.dtype, (P, W - 1, C))
        if slot is None and P < N:
            raise ValueError("conv_state has %d entries for %d sequences" % (P, N))
    elif state_only:
        raise ValueError("state_only needs conv_state")
    for name, t in (("slot", slot), ("has_state", has_state), ("accepted", accepted)):
        if t is not None:
            _flat(name, t, torch.int32, (N,))
    _status(device_status)
    out_stride = (0, 0)
    if state_only:
        out = None
    else:
        if out is None:
            with _on_stream(stream, x):
                out = torch.empty(shape, dtype=x.dtype, device=x.device)
        else:
            _need_cuda("out", out, x.dtype)
            if out.shape != shape or out.stride(-1) != 1:
                raise ValueError("out must have x's shape and a channel dim of stride 1")
        os = out.stride()
        out_stride = (0, os[0]) if cu_seqlens is not None else (os[0], os[1])
    a = ShortConvArgs(x.data_ptr(), _addr(out), weight.data_ptr(), _addr(bias), _addr(conv_state), _addr(slot),
                      _addr(has_state), _addr(accepted), _addr(cu_seqlens), _addr(device_status), *x_stride,
                      *out_stride, N, T, C, norm_channels, P, W, dtype, weight_dtype, 1 if silu else 0, norm_eps)
    st = _fn().kda_short_conv(ctypes.byref(a), _stream_handle(stream))
    if st:
        raise KdaError(st)
    return out


def _heads(name, t, dim, batched, dtype=None):
    """(batch, token, head) strides of a [T, H, D] or [B, T, H, D] tensor."""
    if dtype is not None:
        _need_cuda(name, t, dtype)
    s = t.stride()
    if t.dim() != (4 if batched else 3) or t.shape[-1] != dim or s[-1] != 1:
        raise ValueError("%s must be %s with a channel dim of stride 1"
                         % (name, "[B, T, H, %d]" % dim if batched else "[T, H, %d]" % dim))
    return s[:3] if batched else (0, s[0], s[1])


def _cache(name, t, heads, dim, dtype):
    _need_cuda(name, t, dtype)
    if t.dim() != 4 or t.shape[2] != heads or t.shape[3] != dim or t.stride(3) != 1:
        raise ValueError("%s must be [pages, page_size, %d, %d] with a channel dim of stride 1" % (name, heads, dim))
    return t.stride()[:3]


_NONE3 = (0, 0, 0)


def kda_qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, norm=True, norm_eps=1e-6,
                     interleaved=False, rope_scale=1.0, q_out=None, k_out=None, v=None, k_cache=None, v_cache=None,
                     slots=None, device_status=None, stream=None):
    """RMS norm of every query and key head and the position rotation in one
    pass (see kda_qk_norm_rope in include/kda_ops.h).

    q [T, Hq, D] and k [T, Hk, D] (or [B, T, H, D]) bf16 or fp16; positions int32
    [T] ([B, T]); inv_freq fp32 [rot_dim / 2] (rope_frequencies) or None for the
    norm alone; weights [D] in q's type or fp32 (None: ones); norm=False
    rotates only.  With k_cache [pages, page_size, Hk, D] and slots int64 [T]
    (page * page_size + row, negative: none) the keys go to the cache, and v to
    v_cache; keys are then returned only if k_out is given.  q_out and k_out may
    be q and k themselves.  Returns (q_out, k_out).
    """
    dtype = _elem("q", q)
    batched, dim, dt = q.dim() == 4, q.shape[-1], q.dtype
    qs = _heads("q", q, dim, batched)
    ks = _heads("k", k, dim, batched, dt)
    lead = q.shape[:-2]
    if k.shape[:-2] != lead:
        raise ValueError("q and k must have the same tokens")
    Hq, Hk = q.shape[-2], k.shape[-2]
    B, T = (lead[0], lead[1]) if batched else (1, lead[0])
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.shape[0]
        _flat("inv_freq", inv_freq, torch.float32, (rot // 2,))
        _flat("positions", positions, torch.int32, tuple(lead))
    wq, wk = _weight("q_weight", q_weight, dt, (dim,)), _weight("k_weight", k_weight, dt, (dim,))
    if q_weight is not None and k_weight is not None and wq != wk:
        raise TypeError("q_weight and k_weight must have the same type")
    weight_dtype = wk if q_weight is None else wq
    vs = kcs = vcs = _NONE3
    pages = page_size = 0
    if k_cache is not None:
        kcs = _cache("k_cache", k_cache, Hk, dim, dt)
        pages, page_size = k_cache.shape[0], k_cache.shape[1]
        if slots is None:
            raise ValueError("k_cache needs slots")
        _flat("slots", slots, torch.int64, tuple(lead))
        if v_cache is not None:
            vcs = _cache("v_cache", v_cache, Hk, dim, dt)
            if v is None or v.shape != k.shape or v_cache.shape[:2] != k_cache.shape[:2]:
                raise ValueError("v_cache needs v of k's shape and k_cache's pages")
            vs = _heads("v", v, dim, batched, dt)
    elif slots is not None or v_cache is not None:
        raise ValueError("slots and v_cache need k_cache")
    _status(device_status)
    with _on_stream(stream, q):
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dt, device=q.device)
        if k_out is None and k_cache is None:
            k_out = torch.empty(k.shape, dtype=dt, device=k.device)
    qos = _heads("q_out", q_out, dim, batched, dt)
    kos = _NONE3
    if q_out.shape != q.shape or (k_out is not None and k_out.shape != k.shape):
        raise ValueError("q_out and k_out must have the shapes of q and k")
    if k_out is not None:
        kos = _heads("k_out", k_out, dim, batched, dt)
    a = QkNormRopeArgs(q.data_ptr(), k.data_ptr(), _addr(v) if v_cache is not None else None, q_out.data_ptr(),
                       _addr(k_out), _addr(k_cache), _addr(v_cache), _addr(slots), _addr(positions), _addr(inv_freq),
                       _addr(q_weight), _addr(k_weight), _addr(device_status), *qs, *ks, *vs, *qos, *kos, *kcs, *vcs,
                       B, T, Hq, Hk, dim, rot, pages, page_size, dtype, weight_dtype, 1 if norm else 0,
                       1 if interleaved else 0, norm_eps, rope_scale)
    st = _fn().kda_qk_norm_rope(ctypes.byref(a), _stream_handle(stream))
    if st:
        raise KdaError(st)
    return q_out, k_out


def rope_frequencies(rot_dim, *, base=10000.0, scaling=None, factor=1.0, original_context=None, fast_turns=32.0,
                     slow_turns=1.0, device="cuda"):
    """(inv_freq, rope_scale) for kda_qk_norm_rope.

    inv_freq[i] = base^(-2 i / rot_dim), i < rot_dim / 2, formed in fp64; scaled
    for contexts longer than the `original_context` a model was trained on by
      "linear"   every frequency divided by `factor` (position interpolation);
      "ntk"      the base raised to base * factor^(rot_dim / (rot_dim - 2)), which
                 keeps the fastest frequency and divides the slowest by factor;
      "by_parts" the frequencies that make at least fast_turns turns over
                 original_context kept, those below slow_turns divided by
                 factor, a linear ramp between them (in the index i), and
                 rope_scale = 0.1 ln(factor) + 1 (the NTK-by-parts and attention
                 temperature of Peng et al., "YaRN", 2023).
    """
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if not original_context:
            raise ValueError("by_parts needs original_context")

        def index(turns):   # of the frequency that makes `turns` turns over the original context
            return rot_dim * math.log(original_context / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        low = max(math.floor(index(fast_turns)), 0)
        high = min(math.ceil(index(slow_turns)), rot_dim // 2 - 1)
        keep = 1.0 - ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq / factor * (1.0 - keep) + freq * keep
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'by_parts'")
    return freq.to(torch.float32).to(device), scale


def tree_mask(parents):
    """Mask words for kda_tree_attention from the trees' parents.

    parents: int tensor [R, N]; parents[r, i] < i is the node that node i
    follows, -1 for a node right behind the context, -2 for a node that is not
    in the tree (it sees nothing, not even itself).  Returns int64
    [R, N, ceil(N/64)] on the same device: bit j of row i (bit j mod 64 of word
    j // 64) is set for i itself and its ancestors.
    """
    R, N = parents.shape
    sees = torch.eye(N, dtype=torch.bool, device=parents.device).expand(R, N, N).clone()
    for i in range(N):
        up = parents[:, i].long()
        above = torch.gather(sees, 1, up.clamp_min(0)[:, None, None].expand(R, 1, N))[:, 0]
        sees[:, i] = (sees[:, i] | (above & (up >= 0)[:, None])) & (up >= -1)[:, None]
    words = (N + 63) // 64
    bits = torch.nn.functional.pad(sees, (0, 64 * words - N)).view(R, N, words, 64).long()
    return (bits << torch.arange(64, device=parents.device)).sum(-1)


def kda_tree_attention(q, k_cache, v_cache, page_table, context_lens, *, tree_mask=None, num_nodes=None, scale=None,
                       max_context=None, out=None, return_lse=False, workspace=None, device_status=None, stream=None):
    """Attention of drafted tokens over a paged cache (see kda_tree_attention in
    include/kda_ops.h).

    q [R, N, Hq, D] bf16 or fp16; caches [pages, page_size, Hk, D]; page_table
    int32 [R, pages_per_request]; context_lens int32 [R].  The keys and values
    of request r's N nodes follow its context in the cache.  tree_mask int64
    [R, N, ceil(N/64)]: which nodes a node sees besides the whole context
    (tree_mask(parents); None: a chain, N = 1 a single token); num_nodes int32
    [R]: nodes in use; scale defaults to D^-0.5; max_context: a host upper bound
    of context_lens (None: what the page table can address).  Returns out, or
    (out, lse) with lse fp32 [R, N, Hq].
    """
    dtype = _elem("q", q)
    dt = q.dtype
    if q.dim() != 4:
        raise ValueError("q must be [R, N, Hq, D]")
    R, N, Hq, D = q.shape
    qs = q.stride()
    if qs[3] != 1:
        raise ValueError("the channel (last) dim must have stride 1")
    Hk = k_cache.shape[2]
    kcs = _cache("k_cache", k_cache, Hk, D, dt)
    vcs = _cache("v_cache", v_cache, Hk, D, dt)
    if k_cache.shape[:2] != v_cache.shape[:2]:
        raise ValueError("k_cache and v_cache must have the same pages")
    _need_cuda("page_table", page_table, torch.int32)
    if page_table.dim() != 2 or page_table.shape[0] != R or page_table.stride(1) != 1:
        raise ValueError("page_table must be int32 [R, pages] with contiguous rows")
    _flat("context_lens", context_lens, torch.int32, (R,))
    if num_nodes is not None:
        _flat("num_nodes", num_nodes, torch.int32, (R,))
    if tree_mask is not None:
        _flat("tree_mask", tree_mask, torch.int64, (R, N, (N + 63) // 64))
    _status(device_status)
    lse = None
    with _on_stream(stream, q):
        if out is None:
            out = torch.empty(q.shape, dtype=dt, device=q.device)
        else:
            _need_cuda("out", out, dt)
            if out.shape != q.shape or out.stride(3) != 1:
                raise ValueError("out must have q's shape and a channel dim of stride 1")
        if return_lse:
            lse = torch.empty((R, N, Hq), dtype=torch.float32, device=q.device)
    a = TreeAttentionArgs(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), _addr(lse),
                          page_table.data_ptr(), context_lens.data_ptr(), _addr(num_nodes), _addr(tree_mask), None,
                          _addr(device_status), 0, *qs[:3], *out.stride()[:3], *kcs, *vcs, page_table.stride(0), R, N,
                          Hq, Hk, D, k_cache.shape[0], k_cache.shape[1], page_table.shape[1],
                          0 if max_context is None else max_context, dtype, D ** -0.5 if scale is None else scale)
    L = _fn()
    if workspace is None:
        need = L.kda_tree_attention_workspace_size(ctypes.byref(a))
        if need:
            with _on_stream(stream, q):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _need_cuda("workspace", workspace, torch.uint8)
    if workspace is not None:
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    st = L.kda_tree_attention(ctypes.byref(a), _stream_handle(stream))
    if st:
        raise KdaError(st)
    return (out, lse) if return_lse else out

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
import struct

import torch

from .kda import KdaError, _need_cuda, _on_stream, lib

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


def _packer(args):
    """struct packer of the same layout (native alignment, padded to the size)."""
    code = {_p: "P", _i64: "q", _i32: "i", _f32: "f", ctypes.c_size_t: "N"}
    fmt = "@" + "".join(code[t] for _, t in args._fields_)
    return struct.Struct(fmt + "x" * (ctypes.sizeof(args) - struct.calcsize(fmt))).pack


# A call packs its arguments into bytes at once, which costs a fifth of filling
# a ctypes structure field by field; for a single token the call is the host's time.
_pack_conv, _pack_rope, _pack_tree = _packer(ShortConvArgs), _packer(QkNormRopeArgs), _packer(TreeAttentionArgs)
_funcs = None


def _fn():
    global _funcs
    if _funcs is None:
        L = lib()
        for name in ("kda_short_conv", "kda_qk_norm_rope", "kda_tree_attention"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [_p, _p]
        L.kda_tree_attention_workspace_size.restype = ctypes.c_size_t
        L.kda_tree_attention_workspace_size.argtypes = [_p]
        _funcs = L
    return _funcs


def _raw_stream(stream, like):
    return torch._C._cuda_getCurrentRawStream(like.get_device()) if stream is None else stream.cuda_stream


def _new(stream, like, shape, dtype=None):
    """An uninitialised tensor that belongs to the stream the kernels run on."""
    if stream is None:
        return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)
    with _on_stream(stream, like):
        return like.new_empty(shape, dtype=dtype or like.dtype)


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _elem(name, t):
    """KDA_DTYPE_* of a bf16 or fp16 CUDA tensor."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be bf16 or fp16, got %s" % (name, t.dtype))
    return code


def _flat(name, t, dtype, shape):
    """Address of a contiguous CUDA tensor of one type and shape (None: 0)."""
    if t is None:
        return 0
    if t.dtype is not dtype or not t.is_cuda:
        _need_cuda(name, t, dtype)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous of shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _status(t):
    if t is not None:
        _need_cuda("device_status", t, torch.int32)
    return _addr(t)


def _weight_type(*named):
    """KDA_DTYPE_* of weights that are fp32 or of the data's type, all alike."""
    types = {t.dtype for t in named if t is not None}
    if len(types) > 1:
        raise TypeError("the weights must have the same type")
    return KDA_DTYPE_F32 if not types or torch.float32 in types else _DTYPES.get(types.pop(), -1)


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
    dtype, dt = _elem("x", x), x.dtype
    shape, xs = x.shape, x.stride()
    if len(shape) != (3 if cu_seqlens is None else 2) or xs[-1] != 1:
        raise ValueError("x must be [T_total, C] with cu_seqlens, [B, T, C] without, its last stride 1")
    C = shape[-1]
    if cu_seqlens is None:
        N, T, x0, x1 = shape[0], shape[1], xs[0], xs[1]
    else:
        N, T, x0, x1 = cu_seqlens.shape[0] - 1, shape[0], 0, xs[0]
    if weight.dim() != 2:
        raise ValueError("weight must be [C, W]")
    W = weight.shape[1]
    wt = weight.dtype
    P = 0
    if conv_state is not None:
        P = conv_state.shape[0]
        if slot is None and P < N:
            raise ValueError("conv_state has %d entries for %d sequences" % (P, N))
    elif state_only:
        raise ValueError("state_only needs conv_state")
    o0 = o1 = 0
    if state_only:
        out = None
    else:
        if out is None:
            out = _new(stream, x, shape)
        else:
            _need_cuda("out", out, dt)
            if out.shape != shape or out.stride(-1) != 1:
                raise ValueError("out must have x's shape and a channel dim of stride 1")
        os = out.stride()
        o0, o1 = (os[0], os[1]) if cu_seqlens is None else (0, os[0])
    a = _pack_conv(x.data_ptr(), _addr(out),
                   _flat("weight", weight, wt if wt is torch.float32 else dt, (C, W)),
                   _flat("bias", bias, torch.float32, (C,)), _flat("conv_state", conv_state, dt, (P, W - 1, C)),
                   _flat("slot", slot, torch.int32, (N,)), _flat("has_state", has_state, torch.int32, (N,)),
                   _flat("accepted", accepted, torch.int32, (N,)),
                   _flat("cu_seqlens", cu_seqlens, torch.int32, (N + 1,)),
                   _status(device_status), x0, x1, o0, o1, N, T, C, norm_channels, P,
                   W, dtype, KDA_DTYPE_F32 if wt is torch.float32 else dtype, 1 if silu else 0, norm_eps)
    st = _fn().kda_short_conv(a, _raw_stream(stream, x))
    if st:
        raise KdaError(st)
    return out


def _heads(name, t, heads_shape, dtype):
    """(batch, token, head) strides of a [T, H, D] or [B, T, H, D] tensor."""
    if t.dtype is not dtype or not t.is_cuda:
        _need_cuda(name, t, dtype)
    s = t.stride()
    if t.shape != heads_shape or s[-1] != 1:
        raise ValueError("%s must have shape %s and a channel dim of stride 1, got %s"
                         % (name, tuple(heads_shape), tuple(t.shape)))
    return (0, s[0], s[1]) if len(s) == 3 else s[:3]


def _cache(name, t, heads, dim, dtype):
    if t.dtype is not dtype or not t.is_cuda:
        _need_cuda(name, t, dtype)
    s, shape = t.stride(), t.shape
    if len(shape) != 4 or shape[2] != heads or shape[3] != dim or s[3] != 1:
        raise ValueError("%s must be [pages, page_size, %d, %d] with a channel dim of stride 1" % (name, heads, dim))
    return s[:3]


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
    dtype, dt = _elem("q", q), q.dtype
    qshape, kshape = q.shape, k.shape
    if len(qshape) not in (3, 4):
        raise ValueError("q must be [T, H, D] or [B, T, H, D]")
    lead, dim, Hq = qshape[:-2], qshape[-1], qshape[-2]
    if kshape[:-2] != lead or kshape[-1] != dim:
        raise ValueError("q and k must have the same tokens and head size")
    Hk = kshape[-2]
    B, T = lead if len(lead) == 2 else (1, lead[0])
    rot = fp = pp = 0
    if inv_freq is not None:
        half = inv_freq.shape[0]
        rot = 2 * half
        fp = _flat("inv_freq", inv_freq, torch.float32, (half,))
        pp = _flat("positions", positions, torch.int32, lead)
    wdt = _weight_type(q_weight, k_weight)
    wt = torch.float32 if wdt == KDA_DTYPE_F32 else dt
    vp = kcp = vcp = sp = 0
    vs = kcs = vcs = _NONE3
    pages = page_size = 0
    if k_cache is not None:
        kcs = _cache("k_cache", k_cache, Hk, dim, dt)
        kcp, pages, page_size = k_cache.data_ptr(), k_cache.shape[0], k_cache.shape[1]
        if slots is None:
            raise ValueError("k_cache needs slots")
        sp = _flat("slots", slots, torch.int64, lead)
        if v_cache is not None:
            vcs = _cache("v_cache", v_cache, Hk, dim, dt)
            if v is None or v_cache.shape != k_cache.shape:
                raise ValueError("v_cache needs v, and k_cache's shape")
            vs = _heads("v", v, kshape, dt)
            vp, vcp = v.data_ptr(), v_cache.data_ptr()
    elif slots is not None or v_cache is not None:
        raise ValueError("slots and v_cache need k_cache")
    if q_out is None:
        q_out = _new(stream, q, qshape)
    if k_out is None and k_cache is None:
        k_out = _new(stream, k, kshape)
    a = _pack_rope(q.data_ptr(), k.data_ptr(), vp, q_out.data_ptr(), _addr(k_out), kcp, vcp, sp, pp, fp,
                   _flat("q_weight", q_weight, wt, (dim,)), _flat("k_weight", k_weight, wt, (dim,)),
                   _status(device_status), *_heads("q", q, qshape, dt),
                   *_heads("k", k, kshape, dt), *vs, *_heads("q_out", q_out, qshape, dt),
                   *(_NONE3 if k_out is None else _heads("k_out", k_out, kshape, dt)), *kcs, *vcs, B, T, Hq, Hk, dim,
                   rot, pages, page_size, dtype, wdt, 1 if norm else 0, 1 if interleaved else 0, norm_eps, rope_scale)
    st = _fn().kda_qk_norm_rope(a, _raw_stream(stream, q))
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
    dtype, dt = _elem("q", q), q.dtype
    shape, qs = q.shape, q.stride()
    if len(shape) != 4 or qs[3] != 1:
        raise ValueError("q must be [R, N, Hq, D] with a channel dim of stride 1")
    R, N, Hq, D = shape
    cshape, tshape, ts = k_cache.shape, page_table.shape, page_table.stride()
    Hk = cshape[2]
    kcs, vcs = _cache("k_cache", k_cache, Hk, D, dt), _cache("v_cache", v_cache, Hk, D, dt)
    if v_cache.shape != cshape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if page_table.dtype is not torch.int32 or not page_table.is_cuda:
        _need_cuda("page_table", page_table, torch.int32)
    if len(tshape) != 2 or tshape[0] != R or (ts[1] != 1 and tshape[1] > 1):
        raise ValueError("page_table must be int32 [R, pages] with contiguous rows")
    if out is None:
        out = _new(stream, q, shape)
        os = out.stride()
    else:
        _need_cuda("out", out, dt)
        os = out.stride()
        if out.shape != shape or os[3] != 1:
            raise ValueError("out must have q's shape and a channel dim of stride 1")
    lse = _new(stream, q, (R, N, Hq), torch.float32) if return_lse else None
    head = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), _addr(lse), page_table.data_ptr(),
            _flat("context_lens", context_lens, torch.int32, (R,)), _flat("num_nodes", num_nodes, torch.int32, (R,)),
            _flat("tree_mask", tree_mask, torch.int64, (R, N, (N + 63) // 64)))
    tail = (_status(device_status),)
    sizes = (qs[0], qs[1], qs[2], os[0], os[1], os[2], *kcs, *vcs, ts[0], R, N, Hq, Hk, D, cshape[0], cshape[1],
             tshape[1], 0 if max_context is None else max_context, dtype, D ** -0.5 if scale is None else scale)
    L = _fn()
    if workspace is None:
        need = L.kda_tree_attention_workspace_size(_pack_tree(*head, 0, *tail, 0, *sizes))
        wp = 0
        if need:
            workspace = _new(stream, q, (need,), torch.uint8)
            wp = workspace.data_ptr()
    else:
        need = workspace.numel()
        wp = _flat("workspace", workspace, torch.uint8, (need,))
    st = L.kda_tree_attention(_pack_tree(*head, wp, *tail, need, *sizes), _raw_stream(stream, q))
    if st:
        raise KdaError(st)
    return (out, lse) if return_lse else out

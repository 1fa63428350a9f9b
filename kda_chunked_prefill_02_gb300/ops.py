"""The operators in include/kda_ops.h as Python functions.

The operators a serving decoder runs around KDA: the short causal convolution
(`kda_short_conv`), the query / key norm with the position rotation
(`kda_qk_norm_rope`, frequencies from `rope_frequencies`), and the attention of
drafted tokens over a paged cache (`kda_tree_attention`, masks from
`tree_mask`).  The tensors' checks and the calls are in the native binding
csrc/ops_binding.cpp, which also sees to it that a call's tensors are on one
device; the structures below are the C ABI's, for callers of the library itself.  As in kda.py, outputs and workspaces come from torch, any status
other than KDA_OK raises KdaError, and there is no fallback.
"""
import ctypes
import math

import torch

from .kda import KdaError, _check, _overrides_var, lib

KDA_DTYPE_BF16, KDA_DTYPE_F16, KDA_DTYPE_F32 = range(3)

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


class TreeSchedule(ctypes.Structure):
    _fields_ = _fields("i32: kernel ordered cluster launches")


_funcs = None


def _fn():
    """libkda.so with the operators' signatures (C structures by address)."""
    global _funcs
    if _funcs is None:
        L = lib()
        for name in ("kda_short_conv", "kda_qk_norm_rope", "kda_tree_attention"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [_p, _p]
        L.kda_tree_attention_workspace_size.restype = ctypes.c_size_t
        L.kda_tree_attention_workspace_size.argtypes = [_p]
        L.kda_tree_attention_schedule.restype = ctypes.c_int
        L.kda_tree_attention_schedule.argtypes = [_p, ctypes.c_int, _p]
        _funcs = L
    return _funcs


_binding = None


def _native():
    """The native binding (csrc/ops_binding.cpp; raises if it has not been built)."""
    global _binding
    if _binding is None:
        lib()
        try:
            from . import _kda_ops
        except ImportError as e:
            raise RuntimeError("_kda_ops.so is not built; run `python -m kda_chunked_prefill_02_gb300.build` "
                               "(needs nvcc and g++)") from e
        _kda_ops.set_error(KdaError)
        _binding = _kda_ops
    return _binding


def _run(f, stream, args):
    """f on `stream` (results and workspace belong to it) or on the current stream."""
    if stream is None:
        return f(*args)
    with torch.cuda.stream(stream):
        return f(*args)


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
    return _run((_binding or _native()).short_conv, stream,
                (x, weight, bias, conv_state, slot, has_state, cu_seqlens, accepted, silu, norm_channels, norm_eps,
                 out, state_only, device_status))


def kda_qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, norm=True, norm_eps=1e-6,
                     interleaved=False, rope_scale=1.0, q_out=None, k_out=None, v=None, k_cache=None, v_cache=None,
                     slots=None, device_status=None, stream=None):
    """RMS norm of every query and key head and the position rotation in one
    pass (see kda_qk_norm_rope in include/kda_ops.h).

    q [T, Hq, D] and k [T, Hk, D] (or [B, T, H, D]) bf16 or fp16; positions int32
    [T] ([B, T]); inv_freq fp32 [rot_dim / 2] (rope_frequencies) or None for the
    norm alone; weights [D] in q's type or fp32 (None: ones); norm=False
    rotates only and leaves the weights unread.  With k_cache [pages, page_size, Hk, D] and slots int64 [T]
    (page * page_size + row, negative: none) the keys go to the cache, and v to
    v_cache; keys are then returned only if k_out is given.  q_out and k_out may
    be q and k themselves.  Returns (q_out, k_out).
    """
    return _run((_binding or _native()).qk_norm_rope, stream,
                (q, k, positions, inv_freq, q_weight, k_weight, norm, norm_eps, interleaved, rope_scale, q_out, k_out,
                 v, k_cache, v_cache, slots, device_status))


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
        high = min(math.ceil(index(slow_turns)), rot_dim - 1)   # may lie behind the last frequency
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
    in the tree (it sees no node, not even itself; the context it sees, as every
    node does, so that its row is zero only over an empty one).  Returns int64
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
    of context_lens (None: what the page table can address), by which the kernel and
    its cut are chosen: with a table much wider than the contexts give it
    (tree_attention_schedule tells the choice); out may be q itself.  Returns out, or
    (out, lse) with lse fp32 [R, N, Hq].
    """
    given = _overrides_var.get()
    return _run((_binding or _native()).tree_attention, stream,
                (q, k_cache, v_cache, page_table, context_lens, tree_mask, num_nodes, scale, max_context, out,
                 return_lse, workspace, device_status, None if given is None else ctypes.addressof(given)))


def tree_attention_schedule(q, k_cache, page_table, *, scale=None, max_context=None, num_sms=None):
    """How kda_tree_attention cuts a call (kda_tree_attention_schedule): dict(kernel,
    ordered, cluster, launches), kernel "items", "clusters", "line" or "many rows".  Host
    only; the tensors may live anywhere (only their types and shapes are read).  num_sms
    defaults to the current CUDA device's SM count."""
    a = TreeAttentionArgs()
    a.q = a.out = a.k_cache = a.v_cache = a.page_table = a.context_lens = 16   # not followed
    a.dtype = {torch.bfloat16: KDA_DTYPE_BF16, torch.float16: KDA_DTYPE_F16}.get(q.dtype, KDA_DTYPE_F32)
    a.num_requests, a.max_nodes, a.num_q_heads, a.head_dim = q.shape
    a.num_pages, a.page_size, a.num_k_heads, _ = k_cache.shape
    a.pages_per_request = page_table.shape[1]
    a.max_context = max_context or 0
    a.scale = q.shape[3] ** -0.5 if scale is None else scale
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    s = TreeSchedule()
    _check(_fn().kda_tree_attention_schedule(ctypes.byref(a), int(num_sms), ctypes.byref(s)))
    return dict(kernel=("items", "clusters", "line", "many rows")[s.kernel], ordered=bool(s.ordered),
                cluster=s.cluster, launches=s.launches)

"""Host side of the operators in include/kda_ops.h at the edges (no GPU): refusals of the
Python binding, the helpers' formulas, sizes near the ends of their types."""
import ctypes
import math

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from kda_chunked_prefill_02_gb300 import build, ops as o
    build.build()
    o._fn()
    return o


# ---------------------------------------------------------------- tensors on two devices
def _fake(make):
    """Tensors of a device and a shape without memory: what a check may look at."""
    if 0 < torch.cuda.device_count() < 2:
        pytest.skip("one GPU: torch makes a tensor without memory only for a GPU that is there")
    with FakeTensorMode(allow_non_fake_inputs=True):
        return make()


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("arg", ["weight", "bias", "conv_state", "slot", "has_state", "accepted", "out",
                                 "device_status"])
def test_conv_tensors_on_one_device(ops, arg):
    def make():
        d = {a: "cuda:1" if a == arg else "cuda:0" for a in
             ("weight", "bias", "conv_state", "slot", "has_state", "accepted", "out", "device_status")}
        i32 = dict(dtype=torch.int32)
        return (torch.empty(2, 3, 256, dtype=BF16, device="cuda:0"), torch.empty(256, 4, device=d["weight"]),
                dict(bias=torch.empty(256, device=d["bias"]),
                     conv_state=torch.empty(2, 3, 256, dtype=BF16, device=d["conv_state"]),
                     slot=torch.empty(2, device=d["slot"], **i32), has_state=torch.empty(2, device=d["has_state"], **i32),
                     accepted=torch.empty(2, device=d["accepted"], **i32),
                     out=torch.empty(2, 3, 256, dtype=BF16, device=d["out"]),
                     device_status=torch.empty(1, device=d["device_status"], **i32)))
    x, w, kw = _fake(make)
    with pytest.raises(ValueError, match=arg + " is on cuda:1"):
        ops.kda_short_conv(x, w, **kw)


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("arg", ["k", "positions", "inv_freq", "q_weight", "v", "k_cache", "v_cache", "slots", "q_out",
                                 "k_out", "device_status"])
def test_rope_tensors_on_one_device(ops, arg):
    def make():
        def t(name, *shape, dtype=BF16):
            return torch.empty(*shape, dtype=dtype, device="cuda:1" if name == arg else "cuda:0")
        return (t("q", 5, 4, 128), t("k", 5, 2, 128), t("positions", 5, dtype=torch.int32),
                t("inv_freq", 32, dtype=torch.float32),
                dict(q_weight=t("q_weight", 128), v=t("v", 5, 2, 128), k_cache=t("k_cache", 3, 16, 2, 128),
                     v_cache=t("v_cache", 3, 16, 2, 128), slots=t("slots", 5, dtype=torch.int64),
                     q_out=t("q_out", 5, 4, 128), k_out=t("k_out", 5, 2, 128),
                     device_status=t("device_status", 1, dtype=torch.int32)))
    q, k, pos, freq, kw = _fake(make)
    with pytest.raises(ValueError, match=arg + " is on cuda:1"):
        ops.kda_qk_norm_rope(q, k, pos, freq, **kw)


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("arg", ["k_cache", "v_cache", "page_table", "context_lens", "tree_mask", "num_nodes", "out",
                                 "workspace", "device_status"])
def test_tree_tensors_on_one_device(ops, arg):
    def make():
        def t(name, *shape, dtype=BF16):
            return torch.empty(*shape, dtype=dtype, device="cuda:1" if name == arg else "cuda:0")
        i32 = torch.int32
        return (t("q", 2, 3, 4, 128), t("k_cache", 9, 16, 2, 128), t("v_cache", 9, 16, 2, 128),
                t("page_table", 2, 4, dtype=i32), t("context_lens", 2, dtype=i32),
                dict(tree_mask=t("tree_mask", 2, 3, 1, dtype=torch.int64), num_nodes=t("num_nodes", 2, dtype=i32),
                     out=t("out", 2, 3, 4, 128), workspace=t("workspace", 4096, dtype=torch.uint8),
                     device_status=t("device_status", 1, dtype=i32)))
    q, kc, vc, table, ctx, kw = _fake(make)
    with pytest.raises(ValueError, match=arg + " is on cuda:1"):
        ops.kda_tree_attention(q, kc, vc, table, ctx, **kw)


# ---------------------------------------------------------------- results over the queries
PTR = 1 << 20   # never dereferenced: the checks fail first


def _tree_args(ops, **kw):
    a = ops.TreeAttentionArgs()
    a.q = a.k_cache = a.v_cache = a.page_table = a.context_lens = PTR
    a.out = 2 * PTR
    for n in ("q", "out", "k_cache", "v_cache"):
        for i, s in enumerate((8192, 1024, 128)):
            setattr(a, "%s_stride%d" % (n, i), s)
    a.num_requests, a.max_nodes, a.num_q_heads, a.num_k_heads, a.head_dim = 2, 4, 8, 2, 128
    a.num_pages, a.page_size, a.pages_per_request, a.page_table_stride, a.scale = 100, 16, 50, 50, 0.1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_tree_results_over_other_queries_are_refused(ops):
    """out at q's address with other strides would put rows over queries that other CTAs read.
    (What is not refused is asked for its workspace alone, so that nothing can be launched.)"""
    args = lambda **kw: ctypes.byref(_tree_args(ops, pages_per_request=1000, **kw))  # noqa: E731
    run = lambda **kw: ops._fn().kda_tree_attention(args(**kw), None)  # noqa: E731
    size = lambda **kw: ops._fn().kda_tree_attention_workspace_size(args(**kw))  # noqa: E731
    invalid = 1
    for kw in (dict(out_stride0=4096), dict(out_stride1=2048), dict(out_stride2=256)):
        assert run(out=PTR, **kw) == invalid, kw
        assert size(out=PTR, **kw) == 0 and size(**kw) > 0, kw
    assert size(out=PTR) > 0
    # the stride of a dim of size 1 says nothing
    assert size(out=PTR, num_requests=1, out_stride0=4096) > 0


def test_rope_results_over_other_heads_are_refused(ops):
    """The same with q_out at q's address and k_out at k's.  (Only calls that are refused.)"""
    def run(**kw):
        a = ops.QkNormRopeArgs()
        a.q = a.q_out = a.positions = a.inv_freq = PTR
        a.k = a.k_out = 2 * PTR
        for n in ("q", "k", "q_out", "k_out"):
            for i, s in enumerate((4096, 512, 128)):
                setattr(a, "%s_stride%d" % (n, i), s)
        a.batch, a.seqlen, a.num_q_heads, a.num_k_heads, a.head_dim, a.rot_dim = 2, 3, 4, 2, 128, 64
        a.weight_dtype, a.norm, a.norm_eps, a.rope_scale = 2, 1, 1e-6, 1.0
        for k, v in kw.items():
            setattr(a, k, v)
        return ops._fn().kda_qk_norm_rope(ctypes.byref(a), None)

    invalid = 1
    for kw in (dict(q_out_stride0=8192), dict(q_out_stride1=1024), dict(q_out_stride2=256), dict(k_out_stride0=2048),
               dict(k_out_stride1=256), dict(k_out_stride2=256)):
        assert run(**kw) == invalid, kw


@pytest.mark.parametrize("bound", [(1 << 63) - 1, (1 << 63) - 4, 1 << 62, 1 << 31])
def test_tree_bound_of_the_contexts_near_the_end_of_its_type(ops, bound):
    """A bound past what the page table addresses is no bound."""
    size = lambda **kw: ops._fn().kda_tree_attention_workspace_size(ctypes.byref(_tree_args(ops, **kw)))  # noqa: E731
    want = size(pages_per_request=1000)
    assert want > 0 and size(pages_per_request=1000, max_context=bound) == want
    # and refuses nothing: without a GPU the call gets as far as looking for one
    unsupported = 2
    a = _tree_args(ops, pages_per_request=1000, max_context=bound)
    assert ops._fn().kda_tree_attention(ctypes.byref(a), None) != unsupported


# ---------------------------------------------------------------- how tree attention is cut
def _schedule(ops, R, N, Hq, Hk, D, tokens, page=16, num_sms=152, dtype=BF16, **kw):
    empty = lambda *shape: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    return ops.tree_attention_schedule(empty(R, N, Hq, D), empty(10, page, Hk, D), empty(R, tokens // page),
                                       num_sms=num_sms, **kw)


def test_tree_schedule(ops):
    """One clear case of every cut."""
    assert _schedule(ops, 1, 1, 8, 2, 128, 1008) == dict(kernel="clusters", ordered=False, cluster=8, launches=1)
    assert _schedule(ops, 1, 1, 8, 2, 128, 131072)["kernel"] == "line"
    assert _schedule(ops, 400, 1, 8, 2, 128, 4096) == dict(kernel="items", ordered=True, cluster=1, launches=1)
    assert _schedule(ops, 256, 61, 32, 4, 128, 8192) == dict(kernel="many rows", ordered=False, cluster=1, launches=1)
    assert _schedule(ops, 257, 61, 32, 4, 128, 8192)["launches"] == 2
    # the bound of the contexts counts, not the table's width
    assert _schedule(ops, 1, 1, 8, 2, 128, 131072, max_context=1000)["kernel"] == "clusters"
    # pages that are no multiple of 8, and scales that are not above zero, stay with few rows
    assert _schedule(ops, 24, 61, 32, 4, 128, 8190, page=10)["kernel"] != "many rows"
    assert _schedule(ops, 24, 61, 32, 4, 128, 8192, scale=0.0)["kernel"] != "many rows"


def test_tree_schedule_refusals(ops):
    from kda_chunked_prefill_02_gb300 import KdaError
    for kw in (dict(D=96), dict(dtype=torch.float32), dict(N=257), dict(num_sms=0), dict(Hq=7)):
        with pytest.raises(KdaError):
            _schedule(ops, **{**dict(R=2, N=4, Hq=8, Hk=2, D=128, tokens=800), **kw})
    assert _schedule(ops, 0, 4, 8, 2, 128, 800)["launches"] == 0


# ---------------------------------------------------------------- frequencies
def test_frequencies_by_parts_where_all_are_faster_than_slow_turns(ops):
    """A long original context: the ramp ends behind the last frequency, which is then not
    divided by the whole factor."""
    ctx, factor, n = 131072, 16.0, 64
    f, _ = ops.rope_frequencies(2 * n, device="cpu")
    g, _ = ops.rope_frequencies(2 * n, scaling="by_parts", factor=factor, original_context=ctx, device="cpu")
    turns = f.double() * ctx / (2 * math.pi)
    assert bool((turns > 2).all())
    # f makes `turns` turns at index n ln(ctx / (2 pi turns)) / ln base
    index = lambda t: n * math.log(ctx / (2 * math.pi * t)) / math.log(10000.0)  # noqa: E731
    low, high = math.floor(index(32)), math.ceil(index(1))
    assert 0 < low < n - 1 < high
    keep = (1 - (torch.arange(n).double() - low) / (high - low)).clamp(0, 1)
    assert 0.2 < float(keep[-1]) < 0.3
    want = f.double() * (keep + (1 - keep) / factor)
    assert bool(((g.double() / want - 1).abs() < 2 ** -22).all())


# ---------------------------------------------------------------- the C library without Python's binding
def test_library_builds_without_torch(ops, monkeypatch, tmp_path, capsys):
    """A user of the C interface alone needs neither torch nor its headers."""
    import os
    import sys
    from kda_chunked_prefill_02_gb300 import build
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_kda_ops.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setitem(sys.modules, "torch", None)   # import torch: ImportError
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "left out" in capsys.readouterr().err
    assert build.build(binding=False) == build.LIB
    assert not os.path.exists(build.BINDING) and capsys.readouterr().err == ""

"""Host side of chunk attention, the residual stream's norm, pool copies and the commit of
cache rows (no GPU): refusals, devices, structures."""
import ctypes
import math
import os
import subprocess

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

BF16 = torch.bfloat16
PTR = 1 << 20   # never dereferenced: the checks fail first
BAD, NO = 1, 2


@pytest.fixture(scope="module")
def ops():
    from kda_chunked_prefill_02_gb300 import build, ops as o
    build.build()
    o._fn()
    return o


def _set(a, kw):
    for k, v in kw.items():
        assert hasattr(a, k), k
        setattr(a, k, v)
    return a


# ---------------------------------------------------------------- chunk attention
def _chunk_args(ops, **kw):
    a = ops.ChunkAttentionArgs()
    a.q = a.k_cache = a.v_cache = a.page_table = a.context_lens = PTR
    a.out = 2 * PTR
    for n in ("q", "out", "k_cache", "v_cache"):
        for i, s in enumerate((8192, 1024, 128)):
            setattr(a, "%s_stride%d" % (n, i), s)
    a.num_requests, a.seqlen, a.num_q_heads, a.num_k_heads, a.head_dim = 2, 4, 8, 2, 128
    a.num_pages, a.page_size, a.pages_per_request, a.page_table_stride, a.scale = 100, 16, 50, 50, 0.1
    a.max_context = -1
    return _set(a, kw)


def test_chunk_refusals(ops):
    run = lambda **kw: ops._fn().kda_chunk_attention(ctypes.byref(_chunk_args(ops, **kw)), None)  # noqa: E731
    assert ops._fn().kda_chunk_attention(None, None) == BAD
    for kw in (dict(q=None), dict(k_cache=None), dict(v_cache=None), dict(out=None), dict(page_table=None),
               dict(context_lens=None), dict(seqlen=-1), dict(num_requests=-1), dict(num_q_heads=7),
               dict(num_k_heads=0), dict(num_pages=0), dict(page_size=0), dict(pages_per_request=-1),
               dict(scale=math.nan), dict(scale=math.inf),
               dict(out=PTR, out_stride0=4096), dict(out=PTR, out_stride1=2048), dict(out=PTR, out_stride2=256),
               dict(out=PTR, out_stride2=256, cu_seqlens=PTR)):
        assert run(**kw) == BAD, kw
    for kw in (dict(head_dim=96), dict(head_dim=512), dict(dtype=2), dict(q=PTR + 2), dict(out=PTR + 8),
               dict(k_cache=PTR + 8), dict(q_stride1=1020), dict(v_cache_stride0=-8), dict(num_requests=70000),
               dict(pages_per_request=1 << 30), dict(seqlen=1 << 30), dict(page_table_stride=-1)):
        assert run(**kw) == NO, kw
    for kw in (dict(num_requests=0), dict(seqlen=0)):
        assert run(**kw) == 0 and run(cu_seqlens=PTR, **kw) == 0, kw


def test_chunk_workspace_of_what_is_refused(ops):
    size = lambda **kw: ops._fn().kda_chunk_attention_workspace_size(ctypes.byref(_chunk_args(ops, **kw)))  # noqa: E731
    assert ops._fn().kda_chunk_attention_workspace_size(None) == 0
    assert size(head_dim=96) == 0 and size(num_requests=0) == 0 and size(seqlen=0) == 0
    assert size(out=PTR, out_stride0=4096) == 0


def _schedule(ops, R, T, Hq, Hk, D, tokens, page=16, num_sms=152, dtype=BF16, packed=True, **kw):
    empty = lambda *shape: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    q = empty(T, Hq, D) if packed else empty(R, T, Hq, D)
    return ops.chunk_attention_schedule(q, empty(10, page, Hk, D), empty(R, tokens // page), packed=packed,
                                        num_sms=num_sms, **kw)


def test_chunk_schedule(ops):
    """One clear case of either kernel, and what takes the kernel for few rows whatever its size."""
    assert _schedule(ops, 1, 1, 8, 2, 128, 1008) == dict(kernel="rows", ctas=8)
    assert _schedule(ops, 1, 8192, 32, 8, 128, 8192) == dict(kernel="tensor", ctas=152)
    assert _schedule(ops, 4, 2048, 16, 2, 256, 8192, packed=False) == dict(kernel="tensor", ctas=76)
    # the bound of the contexts counts, not the table's width
    assert _schedule(ops, 1, 1, 8, 2, 128, 131072)["kernel"] == "tensor"
    assert _schedule(ops, 1, 1, 8, 2, 128, 131072, max_context=1000)["kernel"] == "rows"
    assert _schedule(ops, 1, 1, 8, 2, 128, 131072, max_context=0)["kernel"] == "rows"
    for kw in (dict(page=10, tokens=8190), dict(scale=0.0), dict(scale=-1.0), dict(Hq=129, Hk=1)):
        assert _schedule(ops, **{**dict(R=1, T=8192, Hq=32, Hk=8, D=128, tokens=8192), **kw})["kernel"] == "rows"


def test_chunk_schedule_refusals(ops):
    from kda_chunked_prefill_02_gb300 import KdaError
    for kw in (dict(D=96), dict(dtype=torch.float32), dict(num_sms=0), dict(Hq=7)):
        with pytest.raises(KdaError):
            _schedule(ops, **{**dict(R=2, T=4, Hq=8, Hk=2, D=128, tokens=800), **kw})
    assert _schedule(ops, 0, 0, 8, 2, 128, 800)["ctas"] == 0


def test_chunk_workspace(ops):
    """The tensor-core kernel's parts: two items a stretch, 256 rows of their values and log-sums."""
    size = lambda **kw: ops._fn().kda_chunk_attention_workspace_size(ctypes.byref(_chunk_args(ops, **kw)))  # noqa: E731
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152
    long = dict(pages_per_request=20000, page_table_stride=20000)
    assert size(**long) == 2 * sms * (16 + 256 * 129 * 4)
    assert size(**long, max_context=100) == 0
    for bound in ((1 << 63) - 1, 1 << 62, 1 << 31):   # no bound
        assert size(**long, max_context=bound) == size(**long)


# ---------------------------------------------------------------- the residual stream's norm
def _norm(ops, **kw):
    a = ops.ResidualNormArgs()
    a.x, a.y, a.gate, a.out, a.x_out, a.weight, a.post_weight = (PTR * i for i in range(1, 8))
    a.x_stride = a.y_stride = a.gate_stride = a.out_stride = a.x_out_stride = 256
    a.tokens, a.channels, a.weight_dtype, a.alpha, a.norm_eps = 5, 256, 2, 1.0, 1e-6
    return ops._fn().kda_residual_norm(ctypes.byref(_set(a, kw)), None)


def test_norm_refusals(ops):
    assert ops._fn().kda_residual_norm(None, None) == BAD
    alone = dict(y=None, x_out=None, gate=None)
    for kw in (dict(x=None), dict(out=None, x_out=None), dict(x_out=None), dict(y=None), dict(alone, x_out=PTR),
               dict(alone, gate=PTR), dict(alone, post_norm=1), dict(alone, out=None), dict(tokens=-1),
               dict(channels=0), dict(norm_eps=-1.0), dict(norm_eps=math.nan), dict(alpha=math.inf),
               dict(out=PTR), dict(out=3 * PTR), dict(out=5 * PTR), dict(x_out=2 * PTR), dict(x_out=3 * PTR),
               dict(out=2 * PTR, out_stride=512), dict(x_out=PTR, x_out_stride=512), dict(out_stride=248),
               dict(x_out_stride=0)):
        assert _norm(ops, **kw) == BAD, kw
    for kw in (dict(channels=252), dict(channels=16392), dict(dtype=2), dict(dtype=3), dict(x_dtype=1),
               dict(weight_dtype=1), dict(x=PTR + 8), dict(y=PTR + 2), dict(gate=PTR + 8), dict(out=PTR + 8),
               dict(x_out=PTR + 4), dict(weight=PTR + 4), dict(post_weight=PTR + 8), dict(x_stride=260),
               dict(y_stride=-256), dict(gate_stride=4), dict(out_stride=300), dict(tokens=1 << 31)):
        assert _norm(ops, **kw) == NO, kw
    assert _norm(ops, tokens=0) == 0


# ---------------------------------------------------------------- pools
def _pool(ops, **kw):
    p = ops.Pool()
    p.data, p.entries, p.rows, p.cols, p.bytes = PTR, 10, 16, 2, 256
    p.stride0, p.stride1, p.stride2 = 16 * 512, 512, 256
    return _set(p, kw)


POOL_BAD = (dict(entries=-1), dict(rows=-1), dict(cols=-1), dict(bytes=-16), dict(data=None))
POOL_NO = (dict(data=PTR + 8), dict(bytes=24), dict(stride0=8), dict(stride1=-512), dict(stride2=260),
           dict(entries=1 << 31), dict(rows=1 << 31), dict(rows=1 << 16, cols=1 << 16), dict(rows=1 << 20, bytes=1 << 20))


def test_copy_refusals(ops):
    def run(pool=None, second=None, **kw):
        pools = (ops.Pool * 2)(_pool(ops, **(pool or {})), _pool(ops, **(second or {})))
        a = ops.PoolCopyArgs()
        a.pools, a.src, a.dst, a.num_pools, a.count = ctypes.addressof(pools), PTR, PTR, 2, 3
        return ops._fn().kda_pool_copy(ctypes.byref(_set(a, kw)), None)

    assert ops._fn().kda_pool_copy(None, None) == BAD
    for kw in (dict(pools=None), dict(src=None), dict(dst=None), dict(num_pools=-1), dict(count=-1)):
        assert run(**kw) == BAD, kw
    for kw in (dict(num_pools=70000), dict(count=70000)):
        assert run(**kw) == NO, kw
    for kw in POOL_BAD:
        assert run(pool=kw) == BAD and run(second=kw) == BAD, kw
    for kw in POOL_NO:
        assert run(pool=kw) == NO and run(second=kw) == NO, kw
    assert run(count=0) == 0 and run(num_pools=0, pools=None) == 0


def test_commit_refusals(ops):
    def run(pool=None, second=None, **kw):
        pools = (ops.Pool * 2)(_pool(ops, **(pool or {})), _pool(ops, **(second or {})))
        a = ops.CacheCommitArgs()
        a.caches, a.num_caches = ctypes.addressof(pools), 2
        a.page_table = a.context_lens = a.path = a.accepted = PTR
        a.page_table_stride, a.num_requests, a.max_path, a.pages_per_request = 50, 3, 8, 50
        return ops._fn().kda_cache_commit(ctypes.byref(_set(a, kw)), None)

    assert ops._fn().kda_cache_commit(None, None) == BAD
    for kw in (dict(caches=None), dict(page_table=None), dict(context_lens=None), dict(path=None), dict(accepted=None),
               dict(num_caches=-1), dict(num_requests=-1), dict(max_path=-1), dict(pages_per_request=-1),
               dict(pool=dict(rows=8, stride0=8192)), dict(pool=dict(cols=0)), dict(second=dict(bytes=0))):
        assert run(**kw) == BAD, kw
    for kw in (dict(num_caches=70000), dict(num_requests=70000), dict(max_path=257), dict(pages_per_request=1 << 31),
               dict(page_table_stride=-1), dict(pages_per_request=1 << 27),
               dict(pool=dict(cols=1 << 10, bytes=1 << 15))):
        assert run(**kw) == NO, kw
    for kw in POOL_BAD:
        assert run(pool=kw) == BAD and run(second=kw) == BAD, kw
    for kw in POOL_NO:
        assert run(pool=kw) == NO and run(second=kw) == NO, kw
    assert run(num_requests=0) == 0 and run(max_path=0) == 0 and run(num_caches=0, caches=None) == 0


# ---------------------------------------------------------------- the Python binding
def _fake(make):
    if 0 < torch.cuda.device_count() < 2:
        pytest.skip("one GPU: torch makes a tensor without memory only for a GPU that is there")
    with FakeTensorMode(allow_non_fake_inputs=True):
        return make()


def _maker(arg):
    return lambda name, *shape, dtype=BF16: torch.empty(*shape, dtype=dtype, device="cuda:1" if name == arg else "cuda:0")


I32 = torch.int32


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("arg", ["k_cache", "v_cache", "page_table", "context_lens", "cu_seqlens", "out", "workspace",
                                 "device_status"])
def test_chunk_tensors_on_one_device(ops, arg):
    def make():
        t = _maker(arg)
        return ([t("q", 7, 4, 128), t("k_cache", 9, 16, 2, 128), t("v_cache", 9, 16, 2, 128),
                 t("page_table", 2, 4, dtype=I32), t("context_lens", 2, dtype=I32)],
                dict(cu_seqlens=t("cu_seqlens", 3, dtype=I32), out=t("out", 7, 4, 128),
                     workspace=t("workspace", 4096, dtype=torch.uint8), device_status=t("device_status", 1, dtype=I32)))
    a, kw = _fake(make)
    with pytest.raises(ValueError, match=arg + " is on cuda:1"):
        ops.kda_chunk_attention(*a, **kw)


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("arg", ["y", "weight", "post_weight", "gate", "out", "x_out"])
def test_norm_tensors_on_one_device(ops, arg):
    def make():
        t = _maker(arg)
        return ([t("x", 5, 256), t("y", 5, 256)],
                dict(weight=t("weight", 256), post_norm=True, post_weight=t("post_weight", 256), gate=t("gate", 5, 256),
                     out=t("out", 5, 256), x_out=t("x_out", 5, 256)))
    a, kw = _fake(make)
    with pytest.raises(ValueError, match=arg + " is on cuda:1"):
        ops.kda_residual_norm(*a, **kw)


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("arg", ["second", "src", "dst", "rows", "device_status"])
def test_copy_tensors_on_one_device(ops, arg):
    def make():
        t = _maker(arg)
        return ([[t("pools", 5, 16, 64), t("second", 5, 16, 64)], t("src", 2, dtype=I32), t("dst", 2, dtype=I32)],
                dict(rows=t("rows", 2, dtype=I32), device_status=t("device_status", 1, dtype=I32)))
    a, kw = _fake(make)
    with pytest.raises(ValueError, match=("pools" if arg == "second" else arg) + " is on cuda:1"):
        ops.kda_pool_copy(*a, **kw)


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("arg", ["second", "page_table", "context_lens", "path", "accepted", "device_status"])
def test_commit_tensors_on_one_device(ops, arg):
    def make():
        t = _maker(arg)
        return ([[t("caches", 5, 16, 64), t("second", 5, 16, 64)], t("page_table", 2, 3, dtype=I32),
                 t("context_lens", 2, dtype=I32), t("path", 2, 8, dtype=I32), t("accepted", 2, dtype=I32)],
                dict(device_status=t("device_status", 1, dtype=I32)))
    a, kw = _fake(make)
    with pytest.raises(ValueError, match=("caches" if arg == "second" else arg) + " is on cuda:1"):
        ops.kda_cache_commit(*a, **kw)


@pytest.mark.filterwarnings("ignore")
def test_shapes_and_types_are_checked(ops):
    t = _maker("")

    def chunk(**kw):
        a = dict(q=t("", 7, 4, 128), k=t("", 9, 16, 2, 128), v=t("", 9, 16, 2, 128), table=t("", 2, 4, dtype=I32),
                 ctx=t("", 2, dtype=I32), cu_seqlens=t("", 3, dtype=I32))
        a.update(kw)
        return lambda: ops.kda_chunk_attention(a["q"], a["k"], a["v"], a["table"], a["ctx"], cu_seqlens=a["cu_seqlens"],
                                               out=a.get("out"))

    def norm(**kw):
        a = dict(x=t("", 5, 256), y=t("", 5, 256))
        a.update(kw)
        return lambda: ops.kda_residual_norm(a.pop("x"), a.pop("y"), **a)

    def copy(**kw):
        a = dict(pools=[t("", 5, 16, 64)], src=t("", 2, dtype=I32), dst=t("", 2, dtype=I32))
        a.update(kw)
        return lambda: ops.kda_pool_copy(a["pools"], a["src"], a["dst"], rows=a.get("rows"))

    def commit(**kw):
        a = dict(c=[t("", 5, 16, 64)], table=t("", 2, 4, dtype=I32), ctx=t("", 2, dtype=I32), path=t("", 2, 8, dtype=I32),
                 acc=t("", 2, dtype=I32))
        a.update(kw)
        return lambda: ops.kda_cache_commit(a["c"], a["table"], a["ctx"], a["path"], a["acc"])

    def cases():
        return [
            (chunk(q=t("", 7, 4, 128, dtype=torch.float32)), TypeError), (chunk(q=t("", 2, 7, 4, 128)), ValueError),
            (chunk(cu_seqlens=None), ValueError), (chunk(k=t("", 9, 16, 2, 64)), ValueError),
            (chunk(v=t("", 8, 16, 2, 128)), ValueError), (chunk(v=t("", 9, 16, 2, 128, dtype=torch.float16)), TypeError),
            (chunk(table=t("", 3, 4, dtype=I32)), ValueError), (chunk(table=t("", 2, 4, dtype=torch.int64)), TypeError),
            (chunk(table=t("", 4, 2, dtype=I32).t()), ValueError), (chunk(ctx=t("", 3, dtype=I32)), ValueError),
            (chunk(ctx=None), TypeError), (chunk(cu_seqlens=t("", 3, dtype=torch.int64)), TypeError),
            (chunk(out=t("", 7, 4, 64)), ValueError), (chunk(q=t("", 7, 128, 4).transpose(1, 2)), ValueError),
            (norm(y=t("", 5, 128)), ValueError), (norm(x=t("", 5, 256, dtype=torch.float16)), TypeError),
            (norm(y=t("", 5, 256, dtype=torch.float32)), TypeError), (norm(weight=t("", 128)), ValueError),
            (norm(weight=t("", 256, dtype=torch.float16)), TypeError), (norm(gate=t("", 4, 256)), ValueError),
            (norm(weight=t("", 256), post_weight=t("", 256, dtype=torch.float32)), TypeError),
            (norm(y=None, post_norm=True), ValueError), (norm(y=None, norm=False), ValueError),
            (norm(y=None, x_out=t("", 5, 256)), ValueError), (norm(out=t("", 5, 256), norm=False), ValueError),
            (norm(x=t("", 5, 256, dtype=torch.float32), y=None), TypeError),
            (norm(x=t("", 3, 4, 256).transpose(0, 1), y=t("", 4, 3, 256)), ValueError),
            (copy(pools=3), TypeError), (copy(pools=[3]), TypeError), (copy(pools=[t("", 5)]), ValueError),
            (copy(src=t("", 2, dtype=torch.int64)), TypeError), (copy(dst=t("", 3, dtype=I32)), ValueError),
            (copy(rows=t("", 1, dtype=I32)), ValueError), (copy(src=t("", 2, 1, dtype=I32)), ValueError),
            (copy(pools=t("", 5, 4, 6, 8, 64)[:, :, ::2, ::2]), ValueError),
            (commit(c=[t("", 5, 16)]), ValueError), (commit(path=t("", 2, 8, dtype=torch.int64)), TypeError),
            (commit(path=t("", 3, 8, dtype=I32)), ValueError), (commit(acc=None), TypeError), (commit(ctx=None), TypeError),
            (commit(table=t("", 4, 2, dtype=I32).t()), ValueError), (commit(path=t("", 8, 2, dtype=I32).t()), ValueError)]
    for i, (call, error) in enumerate(_fake(cases)):
        with pytest.raises(error):
            call()
            raise AssertionError("case %d was taken" % i)


def test_cpu_tensors_are_refused(ops):
    x = torch.zeros(4, 256, dtype=BF16)
    i = torch.zeros(2, dtype=I32)
    for call in (lambda: ops.kda_chunk_attention(x.view(4, 2, 128), x, x, i, i, cu_seqlens=i),
                 lambda: ops.kda_residual_norm(x, x), lambda: ops.kda_pool_copy([x], i, i),
                 lambda: ops.kda_cache_commit([x.view(2, 2, 256)], i.view(2, 1), i, i.view(2, 1), i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_structures_match_the_header(ops, tmp_path):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    parts = (("kda_chunk_attention_args", ops.ChunkAttentionArgs, "scale"),
             ("kda_residual_norm_args", ops.ResidualNormArgs, "norm_eps"), ("kda_pool", ops.Pool, "bytes"),
             ("kda_pool_copy_args", ops.PoolCopyArgs, "count"),
             ("kda_cache_commit_args", ops.CacheCommitArgs, "pages_per_request"))
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "kda_ops.h"\nint main(void) {\n' + "".join(
        'printf("%%zu %%zu\\n", sizeof(%s), offsetof(%s, %s));\n' % (c, c, f) for c, _, f in parts) + "return 0;\n}\n")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-I" + os.path.join(root, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [v for _, st, f in parts for v in (ctypes.sizeof(st), getattr(st, f).offset)]

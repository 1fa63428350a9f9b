"""Host side of the operators in include/kda_ops.h (no GPU): refusals, the
frequency and mask helpers, the workspace query."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from kda_chunked_prefill_02_gb300 import build, ops as o
    build.build()
    o._fn()
    return o


PTR = 1 << 20   # never dereferenced: the checks fail first


def _conv(ops, **kw):
    a = ops.ShortConvArgs()
    a.x, a.out, a.weight = PTR, 2 * PTR, PTR
    a.x_stride0, a.x_stride1 = 1280, 256
    a.out_stride0, a.out_stride1 = 1280, 256
    a.num_seqs, a.seqlen, a.channels, a.width, a.weight_dtype, a.norm_eps = 2, 5, 256, 4, 2, 1e-6
    for k, v in kw.items():
        setattr(a, k, v)
    return ops._fn().kda_short_conv(ctypes.byref(a), None)


def test_conv_refusals(ops):
    bad, no = 1, 2
    assert ops._fn().kda_short_conv(None, None) == bad
    for kw in (dict(x=None), dict(out=None), dict(weight=None), dict(out=PTR), dict(norm_channels=384),
               dict(norm_channels=-128), dict(channels=0), dict(num_seqs=-1), dict(seqlen=-1), dict(norm_eps=-1.0),
               dict(norm_eps=math.nan), dict(conv_state=PTR, pool_size=0), dict(num_seqs=0, cu_seqlens=PTR)):
        assert _conv(ops, **kw) == bad, kw
    for kw in (dict(width=1), dict(width=5), dict(channels=252), dict(norm_channels=64), dict(dtype=2), dict(dtype=3),
               dict(weight_dtype=1), dict(x=PTR + 2), dict(out=PTR + 8), dict(conv_state=PTR + 8, pool_size=2),
               dict(x_stride1=260), dict(out_stride0=1284), dict(x_stride0=-8), dict(seqlen=1 << 31),
               dict(seqlen=1 << 30), dict(channels=1 << 27)):
        assert _conv(ops, **kw) == no, kw
    assert _conv(ops, num_seqs=0) == 0


def _rope(ops, **kw):
    a = ops.QkNormRopeArgs()
    a.q = a.k = a.q_out = a.k_out = a.positions = a.inv_freq = PTR
    for n in ("q", "k", "v", "q_out", "k_out", "k_cache", "v_cache"):
        for i, s in enumerate((4096, 512, 128)):
            setattr(a, "%s_stride%d" % (n, i), s)
    a.batch, a.seqlen, a.num_q_heads, a.num_k_heads, a.head_dim, a.rot_dim = 1, 3, 4, 2, 128, 64
    a.weight_dtype, a.norm, a.norm_eps, a.rope_scale = 2, 1, 1e-6, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return ops._fn().kda_qk_norm_rope(ctypes.byref(a), None)


def test_rope_refusals(ops):
    bad, no = 1, 2
    assert ops._fn().kda_qk_norm_rope(None, None) == bad
    cache = dict(k_cache=PTR, slots=PTR, num_pages=2, page_size=16)
    for kw in (dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(positions=None),
               dict(inv_freq=None), dict(rot_dim=144), dict(rot_dim=-16), dict(batch=-1), dict(num_q_heads=-1),
               dict(norm_eps=-1e-6), dict(rope_scale=math.inf), dict(slots=PTR), dict(cache, slots=None),
               dict(cache, page_size=0), dict(cache, num_pages=0), dict(cache, v_cache=PTR), dict(v_cache=PTR, v=PTR),
               dict(num_q_heads=0, num_k_heads=0)):
        assert _rope(ops, **kw) == bad, kw
    for kw in (dict(head_dim=120), dict(head_dim=272), dict(rot_dim=24), dict(dtype=2), dict(weight_dtype=1),
               dict(q=PTR + 4), dict(k_out=PTR + 8), dict(q_stride1=516), dict(k_stride2=-128),
               dict(cache, k_cache_stride0=20), dict(cache, k_cache=PTR + 2), dict(num_q_heads=70000),
               dict(batch=1 << 20, seqlen=1 << 12)):
        assert _rope(ops, **kw) == no, kw
    assert _rope(ops, seqlen=0) == 0 and _rope(ops, batch=0) == 0


def _tree_args(ops, **kw):
    a = ops.TreeAttentionArgs()
    a.q = a.k_cache = a.v_cache = a.out = a.page_table = a.context_lens = PTR
    for n in ("q", "out", "k_cache", "v_cache"):
        for i, s in enumerate((8192, 1024, 128)):
            setattr(a, "%s_stride%d" % (n, i), s)
    a.num_requests, a.max_nodes, a.num_q_heads, a.num_k_heads, a.head_dim = 2, 4, 8, 2, 128
    a.num_pages, a.page_size, a.pages_per_request, a.page_table_stride, a.scale = 100, 16, 50, 50, 0.1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_tree_refusals(ops):
    run = lambda **kw: ops._fn().kda_tree_attention(ctypes.byref(_tree_args(ops, **kw)), None)  # noqa: E731
    bad, no = 1, 2
    assert ops._fn().kda_tree_attention(None, None) == bad
    for kw in (dict(q=None), dict(k_cache=None), dict(v_cache=None), dict(out=None), dict(page_table=None),
               dict(context_lens=None), dict(max_nodes=0), dict(num_requests=-1), dict(num_q_heads=7),
               dict(num_k_heads=0), dict(num_pages=0), dict(page_size=0), dict(pages_per_request=-1),
               dict(scale=math.nan), dict(scale=math.inf)):
        assert run(**kw) == bad, kw
    for kw in (dict(head_dim=96), dict(head_dim=512), dict(dtype=2), dict(max_nodes=257), dict(q=PTR + 2),
               dict(k_cache=PTR + 8), dict(q_stride1=1020), dict(v_cache_stride0=-8), dict(num_requests=70000),
               dict(pages_per_request=1 << 30)):
        assert run(**kw) == no, kw
    assert run(num_requests=0) == 0


def test_tree_workspace_query(ops):
    size = lambda **kw: ops._fn().kda_tree_attention_workspace_size(ctypes.byref(_tree_args(ops, **kw)))  # noqa: E731
    assert ops._fn().kda_tree_attention_workspace_size(None) == 0
    assert size(head_dim=96) == 0 and size(num_requests=0) == 0
    # contexts of a tile are not cut; a longer context needs at least two partial rows
    # (128 values and their log-sum in fp32) per query row, 2 requests x 4 nodes x 8 heads
    assert size(pages_per_request=4) == 0
    rows = 2 * 4 * 8
    n = size(pages_per_request=1000)
    assert n >= 2 * rows * 129 * 4
    # a bound of the contexts cuts the work as so many pages would
    assert size(pages_per_request=1000, max_context=60) == 0
    assert size(pages_per_request=1000, max_context=1596) == size(pages_per_request=100)


def test_frequencies_unscaled_and_linear(ops):
    f, s = ops.rope_frequencies(64, base=10000.0, device="cpu")
    want = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
    assert s == 1.0 and f.dtype == torch.float32 and all(abs(float(a) - b) <= 2 ** -24 * b for a, b in zip(f, want))
    g, s = ops.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert s == 1.0 and torch.equal(g, f / 4.0)


def test_frequencies_ntk_ends(ops):
    """The fastest frequency stays, the slowest is divided by the factor."""
    f, _ = ops.rope_frequencies(128, device="cpu")
    g, s = ops.rope_frequencies(128, scaling="ntk", factor=8.0, device="cpu")
    assert s == 1.0 and float(g[0]) == 1.0
    assert abs(float(g[-1]) * 8.0 / float(f[-1]) - 1.0) < 1e-6
    assert bool((g[1:] < f[1:]).all())


def test_frequencies_by_parts(ops):
    """Frequencies with 32 turns and more over the original context stay, those
    below one turn are divided, those between lie between."""
    f, _ = ops.rope_frequencies(128, device="cpu")
    g, s = ops.rope_frequencies(128, scaling="by_parts", factor=16.0, original_context=4096, device="cpu")
    assert abs(s - (0.1 * math.log(16.0) + 1.0)) < 1e-12
    turns = f.double() * 4096 / (2 * math.pi)
    fast, slow = turns >= 33.5, turns <= 0.85
    assert fast.any() and slow.any()
    assert torch.equal(g[fast], f[fast])
    assert bool(((g[slow] * 16.0 / f[slow] - 1.0).abs() < 1e-6).all())
    assert bool((g <= f).all()) and bool((g * 16.0 >= f * (1 - 1e-6)).all()) and bool((g[1:] < g[:-1]).all())
    with pytest.raises(ValueError):
        ops.rope_frequencies(128, scaling="by_parts", factor=16.0)
    with pytest.raises(ValueError):
        ops.rope_frequencies(128, scaling="other")


def test_tree_mask_words(ops):
    #   0 - 2 - 3,  1 - 4;  node 5 outside the tree
    m = ops.tree_mask(torch.tensor([[-1, -1, 0, 2, 1, -2]]))
    assert m.shape == (1, 6, 1)
    assert m[0, :, 0].tolist() == [0b1, 0b10, 0b101, 0b1101, 0b10010, 0]
    chain = ops.tree_mask(torch.arange(-1, 129).view(1, 130))
    assert chain.shape == (1, 130, 3)
    for i in (0, 62, 63, 64, 127, 128, 129):
        bits = [(int(chain[0, i, j // 64]) >> (j % 64)) & 1 for j in range(130)]
        assert bits == [1 if j <= i else 0 for j in range(130)]


def test_python_checks(ops):
    x = torch.zeros(2, 3, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.kda_short_conv(x, torch.zeros(256, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ops.kda_qk_norm_rope(x, x, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        ops.kda_tree_attention(x.view(2, 3, 2, 128), x, x, x, x)


def test_struct_sizes_match_the_header(ops, tmp_path):
    """The binding's structures have the header's size and last field's place."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "s.c"
    src.write_text("""#include <stdio.h>
#include "kda_ops.h"
int main(void) {
    printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(kda_short_conv_args), offsetof(kda_short_conv_args, norm_eps),
           sizeof(kda_qk_norm_rope_args), offsetof(kda_qk_norm_rope_args, rope_scale),
           sizeof(kda_tree_attention_args), offsetof(kda_tree_attention_args, scale));
    return 0;
}
""")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-I" + os.path.join(root, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for st, last in ((ops.ShortConvArgs, "norm_eps"), (ops.QkNormRopeArgs, "rope_scale"),
                     (ops.TreeAttentionArgs, "scale")):
        want += [ctypes.sizeof(st), getattr(st, last).offset]
    assert got == want

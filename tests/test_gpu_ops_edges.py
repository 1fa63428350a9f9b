"""The operators of include/kda_ops.h on the GPU at the edges of what their headers allow."""
from fractions import Fraction

import pytest
import torch

import kda_chunked_prefill_02_gb300 as K
from test_gpu_ops import _tree_case
from ops_test_util import conv_reference, rope_reference, tree_reference, within

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


# 2 pi to 50 digits
TWO_PI = "6.2831853071795864769252867665590057683943387987502"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


# ---------------------------------------------------------------- short convolution
def _inversions():
    even = list(range(0, 1401))                  # one token each, two neighbours' bounds the wrong way round
    swapped = even[:700] + [even[701], even[700]] + even[702:]
    return {"skipped by a search": [0, 100, 10, 20, 200],
            "skipped by a search, long": [0, 100000, 10000, 20000, 200000],
            "one pair of many": swapped,
            "long, at the end": [0, 60000, 60001, 60000, 130000],
            "below zero": [0, -5, 50, 200], "past the tokens": [0, 300, 150, 200],
            "from one": [1, 50, 200], "short of the tokens": [0, 50, 199]}


@pytest.mark.parametrize("what", sorted(_inversions()))
@pytest.mark.parametrize("C", [8, 1536])
def test_conv_reports_every_decrease_of_cu_seqlens(what, C):
    """Wherever the tiles' own search looks, a cu_seqlens that does not run from 0 to the
    token count without decreasing is reported; the sorted one of the same length is not."""
    cu = _inversions()[what]
    total = max(200, max(cu[:-1]) if what == "one pair of many" else 0, cu[-1] if cu[-1] > 200 else 0)
    g = _gen(102)
    x, w = _rand(g, (total, C), BF16).cuda(), _rand(g, (C, 4), torch.float32).cuda()
    st = torch.zeros(len(cu) - 1, 3, C, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.kda_short_conv(x, w, conv_state=st, cu_seqlens=_i32(cu).cuda(), device_status=status)
    assert status.item() == 1
    status.zero_()
    good = sorted(min(max(c, 0), total) for c in cu)
    good[0], good[-1] = 0, total
    K.kda_short_conv(x, w, conv_state=st, cu_seqlens=_i32(good).cuda(), device_status=status)
    assert status.item() == 0


MOST = (1 << 31) - 1   # tokens of a call


def test_conv_state_of_a_sequence_in_the_last_tile_of_the_longest_call():
    """Sums of token numbers near 2^31: the tile that holds the last tokens still owns its
    sequence.  x is one row seen 2^31 - 1 times."""
    g = _gen(103)
    row, w = _rand(g, (1, 8), BF16).cuda(), _rand(g, (8, 4), torch.float32).cuda()
    st = _rand(g, (2, 3, 8), BF16).cuda()
    K.kda_short_conv(row.expand(MOST, 8), w, conv_state=st, cu_seqlens=_i32([0, MOST - 5, MOST]).cuda(),
                     state_only=True)
    assert torch.equal(st, row.expand(2, 3, 8))


def test_conv_outputs_of_the_longest_sequence():
    """One sequence of 2^31 - 1 equal tokens: from the fourth on all outputs are equal, up
    to the last, and nothing is written behind them."""
    g = _gen(104)
    row, w = _rand(g, (1, 8), BF16).cuda(), _rand(g, (8, 4), torch.float32).cuda()
    buf = torch.empty(MOST + 4097, 8, dtype=BF16, device="cuda")
    buf[-8192:] = 7.0
    K.kda_short_conv(row.expand(MOST, 8), w, cu_seqlens=_i32([0, MOST]).cuda(), out=buf[:MOST])
    y, bound, _ = conv_reference(row.cpu().expand(6, 8), w.cpu(), starts=[0], lengths=[6])
    within(buf[:6], y, bound)
    assert torch.equal(buf[MOST - 4095:MOST], buf[5:6].expand(4095, 8))
    assert torch.equal(buf[MOST // 2:MOST // 2 + 64], buf[5:6].expand(64, 8))
    assert bool((buf[MOST:] == 7.0).all())


# ---------------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("wdtype", [torch.float32, BF16])
def test_rope_without_the_norm_leaves_the_weights_alone(interleaved, wdtype):
    """norm=False rotates only: a caller may pass its weights all the same, and gets the
    bits of a call without them, in the outputs and in the cache."""
    g = _gen(101)
    T, Hq, Hk, D = 21, 3, 2, 128
    q, k = _rand(g, (T, Hq, D), BF16), _rand(g, (T, Hk, D), BF16)
    wq, wk = _rand(g, (D,), wdtype).cuda(), _rand(g, (D,), wdtype).cuda()
    pos = torch.randint(0, 100000, (T,), generator=g).to(torch.int32)
    freq, _ = K.rope_frequencies(64, device="cpu")
    slots = torch.arange(T).cuda()

    def run(**kw):
        cache = torch.zeros(2, 16, Hk, D, dtype=BF16, device="cuda")
        out = K.kda_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), freq.cuda(), norm=False, interleaved=interleaved,
                                 k_cache=cache, slots=slots, k_out=torch.empty_like(k, device="cuda"), **kw)
        return (*out, cache)

    plain, weighted = run(), run(q_weight=wq, k_weight=wk)
    for a, b in zip(plain, weighted):
        assert torch.equal(a, b)
    within(weighted[0], *rope_reference(q, pos, freq, None, norm=False, interleaved=interleaved))
    within(weighted[1], *rope_reference(k, pos, freq, None, norm=False, interleaved=interleaved))


@pytest.mark.parametrize("lo,hi", [(1 << 22, 1 << 24), ((1 << 24) - 500, (1 << 24) + 500), (1 << 24, 1 << 31),
                                   (-(1 << 31), -(1 << 24))])
@pytest.mark.parametrize("factor", [1.0, 3.7, 1000.0, 1e6])
def test_rope_angles_of_large_positions_and_frequencies(lo, hi, factor):
    """Products of up to 55 bits, some 3e14 turns.  The reference's angle is formed without
    rounding, from integers, since doubles do not hold it."""
    g = _gen(117)
    T, half = 500, 16
    q = _rand(g, (T, 2, 64), F16)
    pos = torch.randint(lo, hi, (T,), generator=g).to(torch.int32)
    freq = (10000.0 ** (-torch.arange(half).double() / half) * factor).float()
    turn = Fraction(TWO_PI)
    angle = torch.tensor([[float(Fraction(int(p)) * Fraction(float(f)) % turn) for f in freq] for p in pos],
                         dtype=torch.float64)
    out, _ = K.kda_qk_norm_rope(q.cuda(), q.cuda(), pos.cuda(), freq.cuda(), norm=False)
    # the reference with these angles: positions 0 .. T - 1 stand for them one by one
    y = torch.empty(T, 2, 64, dtype=torch.float64)
    bound = torch.empty_like(y)
    for t in range(T):
        y[t:t + 1], bound[t:t + 1] = rope_reference(q[t:t + 1], torch.ones(1), angle[t], None, norm=False)
    within(out, y, bound)


# ---------------------------------------------------------------- tree attention
ROOM = 300000   # tokens a page table has room for: enough for the kernel for many rows


def _tree_inputs(seed, ctx, N, Hq, Hk, D, page, dtype=BF16, room=0):
    """q, caches, table, contexts on the host: every request its own pages."""
    g = _gen(seed)
    need = [(c + N + page - 1) // page for c in ctx]
    table = torch.zeros((len(ctx), max(max(need), room // page)), dtype=torch.int32)
    order, at = torch.randperm(sum(need), generator=g).to(torch.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    kc, vc = _rand(g, (sum(need), page, Hk, D), dtype), _rand(g, (sum(need), page, Hk, D), dtype)
    return _rand(g, (len(ctx), N, Hq, D), dtype), kc, vc, table, _i32(ctx)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,Hq,Hk,room", [(1, 4, 2, 0), (3, 8, 2, 0), (40, 16, 2, 0), (40, 16, 2, ROOM),
                                          (5, 8, 2, ROOM)])
def test_tree_results_over_the_queries(D, N, Hq, Hk, room):
    """out = q: every cut of both kernels, whole items and parts."""
    q, kc, vc, table, ctx = _tree_inputs(105, [3000, 0, 17, 900], N, Hq, Hk, D, 16, room=room)
    out, ob, _, _ = tree_reference(q, kc, vc, table, ctx)
    dev = [t.cuda() for t in (kc, vc, table, ctx)]
    qd = q.cuda()
    apart = K.kda_tree_attention(qd, *dev)
    assert torch.equal(qd.cpu(), q)
    over = K.kda_tree_attention(qd, *dev, out=qd)
    assert over is qd
    within(over, out, ob)
    if D != 256:   # the same kernel as apart from the queries: the same bits
        assert torch.equal(over, apart)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("gap", [13.0, 17.5, 20.0])
@pytest.mark.parametrize("N,Hq,D,kernel", [(1, 2, 64, "items"), (2, 2, 128, "items"), (1, 2, 256, "items"),
                                           (20, 2, 64, "many rows"), (20, 2, 128, "many rows"),
                                           (20, 2, 256, "many rows"), (100, 2, 128, "many rows")])
def test_tree_weight_in_many_keys_far_below_the_largest(dtype, gap, N, Hq, D, kernel):
    """One key whose score is `gap` above all others' and whose value is 0, before 200000 keys
    with values near 1: the result is the many keys' share, 200000 e^-gap of the whole.  As
    many equal requests as make a CTA take a context whole.  A weight's rounding to fp16 is
    off by its unit, or where it is smaller by half of 2^-24 at the kernels' scales (2^11 at
    least)."""
    g = _gen(114)
    L, R, page = 200000, 4 * 160, 16
    q, kc, vc, table, ctx = _tree_inputs(115, [L], N, Hq, 1, D, page, dtype, room=ROOM)
    q[:], kc[:] = 0, 0
    q[..., 0] = 1.0
    vc.copy_(1 + _rand(g, vc.shape, torch.float32, 0.1))
    at = int(table[0, 77])
    kc[at, 5, 0, 0], vc[at, 5] = gap, 0
    # the nodes differ in the last keys that they see, N of 200000: one node stands for all
    out, ob, lse, lb = tree_reference(q[:, -1:], kc, vc, table, ctx + N - 1, scale=1.0)
    ob, lb = ob + out.abs() * N / L, lb + N / L
    if dtype == F16:
        ob = ob + (L + N) * 2.0 ** -25 * 2.0 ** -11 * vc.abs().max().double()
    dev = [t.cuda() for t in (q.expand(R, N, Hq, D).contiguous(), kc, vc, table.expand(R, table.shape[1]).contiguous(),
                              ctx.expand(R).contiguous())]
    assert K.tree_attention_schedule(dev[0], dev[1], dev[3], scale=1.0)["kernel"] == kernel
    got, glse = K.kda_tree_attention(*dev, scale=1.0, return_lse=True)
    for r in (0, 1, R // 2, R - 1):
        within(got[r], out[0].expand(N, Hq, D), ob[0].expand(N, Hq, D))
        within(glse[r], lse[0].expand(N, Hq), lb[0].expand(N, Hq))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scale", [1e-38, 1e-20, 1e10])
def test_tree_scales_near_the_ends_of_their_type(dtype, scale):
    """Every key alike, and one key alone, through the rows that would take the kernel for many."""
    _tree_case(116, [900, 64, 0], 12, 8, 2, 128, 16, dtype, scale=scale, room=ROOM, q_scale=1.0 if scale < 1 else 1e-10)


def _cut(ctx, N, Hq, Hk, D, page, room):
    """How _tree_case's call is cut on this GPU."""
    empty = lambda *shape: torch.empty(shape, dtype=BF16, device="meta")  # noqa: E731
    width = max(max((c + N + page - 1) // page for c in ctx), 1, room // page)
    return K.tree_attention_schedule(empty(len(ctx), N, Hq, D), empty(1, page, Hk, D), empty(len(ctx), width))


@pytest.mark.parametrize("D,N,Hq,Hk", [(64, 9, 4, 2), (128, 34, 16, 2), (256, 20, 4, 2)])
def test_tree_more_requests_than_a_launch_of_the_kernel_for_many_rows(D, N, Hq, Hk):
    """Two launches, the second over the requests from 256 on in the same workspace: one and
    two row tiles, most contexts short, some empty, some long enough to be cut, in both."""
    ctx = [(i * 37) % 90 if i % 50 else 700 + 9 * i for i in range(300)]
    nodes = _i32([(i * 7) % (N + 1) for i in range(300)])
    cut = _cut(ctx, N, Hq, Hk, D, 16, ROOM)
    assert cut["kernel"] == "many rows" and cut["launches"] == 2
    _tree_case(110, ctx, N, Hq, Hk, D, 16, BF16, nodes=nodes, room=ROOM)


@pytest.mark.parametrize("D,R,N,Hk", [(64, 330, 1, 2), (64, 220, 3, 3), (128, 170, 3, 2), (256, 160, 1, 1)])
def test_tree_more_items_than_run_at_once(D, R, N, Hk):
    """A CTA an item, the requests longest first."""
    ctx = [(i * 37) % 90 if i % 50 else 700 + i for i in range(R)]
    nodes = _i32([(i * 7) % (N + 1) for i in range(R)])
    cut = _cut(ctx, N, 2 * Hk, Hk, D, 16, 0)
    assert cut["kernel"] == "items" and cut["ordered"]
    _tree_case(111, ctx, N, 2 * Hk, Hk, D, 16, BF16, nodes=nodes)


# ---------------------------------------------------------------- waits that run out
KDA_ERR_TIMEOUT = 4


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,Hq,ctx", [(24, 4, [3000, 0, 900, 17]),             # one row tile: two streams over one item
                                      (40, 16, [20000, 5, 300, 700] * 20)])    # two row tiles, many items a CTA
def test_tree_wait_that_runs_out_is_reported_and_the_context_survives(D, N, Hq, ctx):
    """The first wait of the softmax warps is for a barrier that nothing arrives on, so that it
    runs out with copies and products in flight.  The call returns and says so, and the next
    one on the same stream and workspace gives the usual bits."""
    pages = 4000   # the requests share them
    kc = torch.randn(pages, 16, 2, D, device="cuda").to(BF16)
    vc = torch.randn_like(kc)
    g = _gen(108)
    table = torch.randint(0, pages, (len(ctx), ROOM // 16), generator=g).to(torch.int32).cuda()
    q, lens = _rand(g, (len(ctx), N, Hq, D), BF16).cuda(), _i32(ctx).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    usual = K.kda_tree_attention(q, kc, vc, table, lens, device_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for limit in (2000, 200000):
        with K.overrides(wait_limit_ns=limit, timeout_probe=True):
            K.kda_tree_attention(q, kc, vc, table, lens, device_status=status)
        torch.cuda.synchronize()            # returns: no hang, no fault
        assert status.item() == KDA_ERR_TIMEOUT
        status.zero_()
        again = K.kda_tree_attention(q, kc, vc, table, lens, device_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0 and torch.equal(again, usual)


def test_tree_waits_that_last_as_long_as_an_item_do_not_run_out():
    """Some roles wait for an item's last tile from its first on, or for a free place among the
    items dealt out.  An item of 8192 key tiles takes a CTA some 16 ms; the bound of a wait
    here is 1 ms beside what the contexts themselves may take."""
    g = _gen(109)
    R, pages = 38, 600   # the requests share their pages
    kc, vc = (torch.randn(pages, 64, 4, 128, device="cuda").to(BF16) for _ in range(2))
    table = torch.randint(0, pages, (R, (1 << 14) + 1), generator=g).to(torch.int32).cuda()
    q, lens = _rand(g, (R, 32, 32, 128), BF16).cuda(), torch.full((R,), 1 << 20, dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    usual = K.kda_tree_attention(q, kc, vc, table, lens)
    with K.overrides(wait_limit_ns=1000000):
        got = K.kda_tree_attention(q, kc, vc, table, lens, device_status=status)
    assert status.item() == 0 and torch.equal(got, usual)


# ---------------------------------------------------------------- strides of dims of size 1
def test_one_token_as_a_transposed_column():
    """The row of a transposed column has strides (1, 1): what a matrix times a column
    leaves behind.  Every operator takes it as the contiguous row that it is."""
    g = _gen(106)

    def row(n):
        r = _rand(g, (n, 1), BF16).cuda().t()
        assert r.stride() == (1, 1) and r.is_contiguous()
        return r

    x = row(384)
    w = _rand(g, (384, 4), torch.float32).cuda()
    cu = _i32([0, 1]).cuda()
    st = [torch.zeros(1, 3, 384, dtype=BF16, device="cuda") for _ in range(3)]
    want = K.kda_short_conv(x.as_strided((1, 384), (384, 1)), w, conv_state=st[0], cu_seqlens=cu, norm_channels=256)
    res = row(384)
    assert torch.equal(K.kda_short_conv(x, w, conv_state=st[1], cu_seqlens=cu, norm_channels=256), want)
    batch = ((1, 1, 384), (1, 1, 1))
    K.kda_short_conv(x.as_strided(*batch), w, conv_state=st[2], norm_channels=256, out=res.as_strided(*batch))
    assert torch.equal(res, want)
    assert torch.equal(st[1], st[0]) and torch.equal(st[2], st[0])

    qkv = row(8 * 128).as_strided((1, 8, 128), (1, 128, 1))
    freq, _ = K.rope_frequencies(128)
    pos = _i32([5]).cuda()
    q, k = K.kda_qk_norm_rope(qkv[:, :6], qkv[:, 6:], pos, freq)
    same = qkv.as_strided((1, 8, 128), (1024, 128, 1))
    q2, k2 = K.kda_qk_norm_rope(same[:, :6], same[:, 6:], pos, freq)
    assert torch.equal(q, q2) and torch.equal(k, k2)

    for N, room in ((1, 0), (24, ROOM)):
        q, kc, vc, table, ctx = _tree_inputs(107, [200], N, 4, 2, 128, 16, room=room)
        dev = [t.cuda() for t in (kc, vc, table, ctx)]
        qd = q.cuda()
        odd = qd.as_strided(qd.shape, (1, *qd.stride()[1:]))
        assert torch.equal(K.kda_tree_attention(odd, *dev), K.kda_tree_attention(qd, *dev))

"""The operators of include/kda_ops.h on the GPU against their 64-bit forms."""
import math

import pytest
import torch

import kda_chunked_prefill_02_gb300 as K
from ops_test_util import conv_reference, rope_reference, tree_reference, within

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _dev(t):
    return None if t is None else t.cuda()


# ---------------------------------------------------------------- short convolution
def _conv_case(seed, lengths, C, W, dtype, *, packed=True, norm=0, bias=False, silu=True, wdtype=torch.float32,
               state=True, has=None, slots=None, accepted=None, pool=None):
    g = _gen(seed)
    total = sum(lengths)
    x = _rand(g, (total, C), dtype)
    w = _rand(g, (C, W), wdtype, W ** -0.5)
    b = _rand(g, (C,), torch.float32, 0.3) if bias else None
    n = len(lengths)
    pool = pool or n
    st = _rand(g, (pool, W - 1, C), dtype) if state else None
    starts = [sum(lengths[:i]) for i in range(n)]
    y, bound, new = conv_reference(x, w, bias=b, state=st, starts=starts, lengths=lengths, slots=slots, has_state=has,
                                   accepted=accepted, silu=silu, norm_channels=norm)
    dst = None if st is None else st.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd = x.cuda()
    cu = None
    if packed:
        cu = _i32(starts + [total]).cuda()
    else:
        xd = xd.view(n, lengths[0], C)
    out = K.kda_short_conv(xd, w.cuda(), bias=_dev(b), conv_state=dst, slot=_dev(slots), has_state=_dev(has),
                           cu_seqlens=cu, accepted=_dev(accepted), silu=silu, norm_channels=norm,
                           device_status=status)
    assert status.item() == 0
    within(out.reshape(total, C), y, bound)
    if st is not None:
        assert torch.equal(dst.cpu(), new)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("C,norm", [(8, 0), (264, 0), (384, 256), (1000, 384), (1536, 1536), (2056, 0)])
def test_conv_packed(W, dtype, C, norm):
    _conv_case(1, [5, 1, 0, 2, 3, 130, 1, 0], C, W, dtype, norm=norm, bias=(W == 3),
               wdtype=dtype if W == 2 else torch.float32)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 65])
def test_conv_padded(tokens, silu):
    _conv_case(2, [tokens] * 3, 768, 4, BF16, packed=False, norm=512, silu=silu)


def test_conv_tiles_meet_many_sequences():
    """Few channels and many tokens: tiles of up to 64 tokens that hold whole short
    sequences, empty ones, and sequences that start a token before a tile's end."""
    lengths = []
    for i in range(700):
        lengths += [63, 1, 0, 62, 2, 0, 0, 1, 127, 3, 5, 64, (i * 37) % 200]
    n = len(lengths)
    perm = torch.randperm(n + 9, generator=_gen(4))[:n].to(torch.int32)
    has = (torch.arange(n) % 3 != 0).to(torch.int32)
    acc = _i32([(length * (i % 4)) // 3 if i % 4 < 3 else length for i, length in enumerate(lengths)])
    _conv_case(3, lengths, 8, 4, BF16, slots=perm, has=has, accepted=acc, pool=n + 9)
    _conv_case(5, lengths, 16, 3, F16, slots=perm, has=has, pool=n + 9, bias=True)


def test_conv_without_a_state():
    _conv_case(6, [4, 70, 1], 256, 4, BF16, norm=128, state=False)


@pytest.mark.parametrize("cut", [1, 2, 3, 40, 129])
def test_conv_pieces_are_the_whole(cut):
    """A prompt in two pieces, then token by token, gives the bits of one call."""
    g = _gen(7)
    x, w = _rand(g, (2, 140, 512), BF16).cuda(), _rand(g, (512, 4), torch.float32).cuda()
    st = torch.zeros(2, 3, 512, dtype=BF16, device="cuda")
    whole = K.kda_short_conv(x, w, conv_state=st, norm_channels=256)
    st2 = torch.zeros_like(st)
    parts = [K.kda_short_conv(x[:, :cut], w, conv_state=st2, norm_channels=256),
             K.kda_short_conv(x[:, cut:135], w, conv_state=st2, norm_channels=256)]
    parts += [K.kda_short_conv(x[:, t:t + 1], w, conv_state=st2, norm_channels=256) for t in range(135, 140)]
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(st, st2)


def test_conv_commit_of_accepted_drafts():
    """Drafts run with accepted 0 (the state stays), then the commit alone."""
    g = _gen(8)
    x, w = _rand(g, (3, 5, 264), F16).cuda(), _rand(g, (264, 4), F16).cuda()
    st = _rand(g, (3, 3, 264), F16).cuda()
    before = st.clone()
    K.kda_short_conv(x, w, conv_state=st, accepted=_i32([0, 0, 0]).cuda())
    assert torch.equal(st, before)
    acc = _i32([0, 2, 5]).cuda()
    assert K.kda_short_conv(x, w, conv_state=st, accepted=acc, state_only=True) is None
    ext = torch.cat([before, x], 1)
    for n, a in enumerate([0, 2, 5]):
        assert torch.equal(st[n], ext[n, a:a + 3])


def test_conv_strided_rows_and_extreme_inputs():
    """x and out as column blocks of wider rows; values where SiLU saturates."""
    g = _gen(9)
    wide = _rand(g, (33, 1024), BF16, 100.0).cuda()
    x = wide[:, 256:768]
    w = _rand(g, (512, 4), torch.float32)
    y, bound, _ = conv_reference(x.cpu(), w, starts=[0], lengths=[33])
    res = torch.full((33, 1024), 7.0, dtype=BF16, device="cuda")
    K.kda_short_conv(x, w.cuda(), cu_seqlens=_i32([0, 33]).cuda(), out=res[:, 512:])
    within(res[:, 512:], y, bound)
    assert bool((res[:, :512] == 7.0).all())


def test_conv_reports_what_only_the_device_sees():
    g = _gen(10)
    x, w = _rand(g, (4, 6, 128), BF16).cuda(), _rand(g, (128, 4), torch.float32).cuda()
    st = _rand(g, (4, 3, 128), BF16).cuda()
    ref_st = st.clone()
    ref = K.kda_short_conv(x, w, conv_state=ref_st)
    for kw, bad in ((dict(slot=_i32([0, 4, 2, 3]).cuda()), 1), (dict(slot=_i32([0, 1, -1, 3]).cuda()), 2),
                    (dict(accepted=_i32([6, 6, 6, 7]).cuda()), 3), (dict(accepted=_i32([-1, 6, 6, 6]).cuda()), 0)):
        s2, status = st.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.zeros_like(x)
        K.kda_short_conv(x, w, conv_state=s2, out=out, device_status=status, **kw)
        assert status.item() == 1
        for n in range(4):
            assert torch.equal(out[n], torch.zeros_like(out[n]) if n == bad else ref[n])
            assert torch.equal(s2[n], st[n] if n == bad else ref_st[n])
    for cu in ([0, 6, 4, 24], [1, 6, 12, 24], [0, 6, 12, 20], [0, 6, 30, 24]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        K.kda_short_conv(x.view(24, 128), w, cu_seqlens=_i32(cu).cuda(), device_status=status)
        assert status.item() == 1, cu


# ---------------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,rot,Hq,Hk", [(128, 128, 8, 2), (128, 64, 5, 3), (64, 64, 3, 1), (64, 16, 16, 16),
                                         (256, 64, 4, 1), (256, 256, 3, 2), (96, 32, 7, 2), (16, 16, 2, 1),
                                         (128, 0, 4, 4), (192, 128, 1, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(dtype, D, rot, Hq, Hk, interleaved):
    g = _gen(D + rot + Hq)
    T = 37
    q, k = _rand(g, (T, Hq, D), dtype, 2.0), _rand(g, (T, Hk, D), dtype, 0.5)
    wq, wk = _rand(g, (D,), torch.float32), _rand(g, (D,), torch.float32)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32)
    pos[:4] = _i32([0, 1, (1 << 24) + 1, (1 << 31) - 1])
    freq, scale = K.rope_frequencies(rot, scaling="by_parts", factor=8.0, original_context=4096, device="cpu") \
        if rot else (None, 1.0)
    qo, ko = K.kda_qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), _dev(freq), q_weight=wq.cuda(), k_weight=wk.cuda(),
                                interleaved=interleaved, rope_scale=scale)
    within(qo, *rope_reference(q, pos, freq, wq, interleaved=interleaved, scale=scale))
    within(ko, *rope_reference(k, pos, freq, wk, interleaved=interleaved, scale=scale))


@pytest.mark.parametrize("T", [1, 2, 300, 5000])
def test_rope_rotation_alone_batched_and_in_place(T):
    g = _gen(T)
    q, k = _rand(g, (2, T, 4, 64), BF16), _rand(g, (2, T, 2, 64), BF16)
    pos = torch.arange(2 * T, dtype=torch.int32).view(2, T)
    freq, _ = K.rope_frequencies(64, device="cpu")
    qd, kd = q.cuda(), k.cuda()
    qo, ko = K.kda_qk_norm_rope(qd, kd, pos.cuda(), freq.cuda(), norm=False, q_out=qd, k_out=kd)
    assert qo is qd and ko is kd
    for got, x in ((qd, q), (kd, k)):
        y, b = rope_reference(x.reshape(2 * T, -1, 64), pos.reshape(-1), freq, None, norm=False)
        within(got.reshape(2 * T, -1, 64), y, b)


@pytest.mark.parametrize("page,heads_first", [(1, False), (16, False), (100, True), (64, True)])
@pytest.mark.parametrize("wdtype", [torch.float32, BF16])
def test_rope_into_a_cache(page, heads_first, wdtype):
    """q, k, v as views of one fused row; keys and values to scattered cache rows
    (negative slots: none), the cache in either order of row and head; nothing
    else in the cache changes."""
    g = _gen(page)
    T, Hq, Hk, D = 83, 6, 3, 128
    qkv = _rand(g, (T, Hq + 2 * Hk, D), BF16)
    pages = (T + page - 1) // page + 2
    pos = torch.randint(0, 200000, (T,), generator=g).to(torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[5] = slots[60] = -1
    freq, _ = K.rope_frequencies(128, base=5e5, device="cpu")
    wq, wk = _rand(g, (D,), wdtype), _rand(g, (D,), wdtype)
    shape = (pages, Hk, page, D) if heads_first else (pages, page, Hk, D)
    kc, vc = _rand(g, shape, BF16).cuda(), _rand(g, shape, BF16).cuda()
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    kc0, vc0 = kc.cpu().clone(), vc.cpu().clone()
    d = qkv.cuda()
    q, k, v = d[:, :Hq], d[:, Hq:Hq + Hk], d[:, Hq + Hk:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, none = K.kda_qk_norm_rope(q, k, pos.cuda(), freq.cuda(), q_weight=wq.cuda(), k_weight=wk.cuda(), v=v,
                                  k_cache=kc, v_cache=vc, slots=slots.cuda(), device_status=status)
    assert none is None and status.item() == 0
    within(qo, *rope_reference(q.cpu(), pos, freq, wq))
    y, b = rope_reference(k.cpu(), pos, freq, wk)
    rows = [(t, int(s) // page, int(s) % page) for t, s in enumerate(slots) if s >= 0]
    for t, p, o in rows:
        within(kc[p, o], y[t], b[t])
        assert torch.equal(vc[p, o].cpu(), v[t].cpu())
        kc0[p, o], vc0[p, o] = kc[p, o].cpu(), vc[p, o].cpu()
    assert torch.equal(kc.cpu(), kc0) and torch.equal(vc.cpu(), vc0)
    # a slot past the cache: reported, skipped, the rest as before; keys also to k_out
    slots[7] = pages * page
    ko = torch.empty(T, Hk, D, dtype=BF16, device="cuda")
    kc1 = kc.clone()
    K.kda_qk_norm_rope(q, k, pos.cuda(), freq.cuda(), q_weight=wq.cuda(), k_weight=wk.cuda(), k_cache=kc,
                       slots=slots.cuda(), k_out=ko, device_status=status)
    assert status.item() == 1 and torch.equal(kc, kc1)
    within(ko, y, b)


def test_rope_channels_that_do_not_rotate_pass():
    q = torch.full((1, 1, 64), 3.0, dtype=BF16)
    q[0, 0, 40] = math.inf
    freq, _ = K.rope_frequencies(32, device="cpu")
    out, _ = K.kda_qk_norm_rope(q.cuda(), q.cuda(), _i32([9]).cuda(), freq.cuda(), norm=False)
    assert torch.equal(out[0, 0, 32:].cpu(), q[0, 0, 32:]) and bool(torch.isfinite(out[0, 0, :32]).all())


def test_rope_zero_rows():
    """A zero head: 0 / sqrt(0 + eps) = 0."""
    z = torch.zeros(2, 2, 128, dtype=BF16, device="cuda")
    freq, _ = K.rope_frequencies(128)
    out, _ = K.kda_qk_norm_rope(z, z, _i32([0, 5]).cuda(), freq)
    assert bool((out == 0).all())


# ---------------------------------------------------------------- tree attention
ROOM = 300000   # tokens a page table has room for: enough for the kernel for many rows


def _pages(g, need_tokens, page, spare=2, room=0):
    need = [(t + page - 1) // page for t in need_tokens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(need), max(max(need), 1, room // page)), 0, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table, total


def _random_parents(g, R, N):
    return (torch.rand((R, N), generator=g) * (torch.arange(N) + 1)).long() - 1


def _sees(parents):
    R, N = parents.shape
    sees = torch.zeros(R, N, N, dtype=torch.bool)
    for r in range(R):
        for i in range(N):
            j = i
            while j >= 0:
                sees[r, i, j] = True
                j = int(parents[r, j])
            if int(parents[r, i]) < -1:
                sees[r, i] = False
    return sees


def _tree_case(seed, ctx, N, Hq, Hk, D, page, dtype, *, form="tree", nodes=None, heads_first=False, q_scale=1.0,
               scale=None, max_context=None, poison=True, parents=None, room=0):
    g = _gen(seed)
    R = len(ctx)
    table, total = _pages(g, [c + N for c in ctx], page, room=room)
    shape = (total, Hk, page, D) if heads_first else (total, page, Hk, D)
    kc, vc = _rand(g, shape, dtype), _rand(g, shape, dtype)
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    q = _rand(g, (R, N, Hq, D), dtype, q_scale)
    if form == "tree" and parents is None:
        parents = _random_parents(g, R, N)
    sees = None if form == "chain" else _sees(parents)
    out, ob, lse, lb = tree_reference(q, kc, vc, table, ctx, sees=sees, nodes=nodes, scale=scale)
    if poison:
        # whatever no request may read holds NaN: spare pages, rows past the end of a
        # page's use, nodes that no row sees
        seen = torch.zeros(total, page, dtype=torch.bool)
        for r in range(R):
            n = N if nodes is None else int(nodes[r])
            keep = [p for p in range(ctx[r] + n)
                    if p < ctx[r] or sees is None or bool(sees[r, :n, p - ctx[r]].any())]
            for p in keep:
                seen[int(table[r, p // page]), p % page] = True
        kc[~seen], vc[~seen] = math.nan, math.nan
    kd, vd = kc.cuda(), vc.cuda()
    if heads_first:
        assert not kd.is_contiguous()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mask = None if sees is None else K.tree_mask(parents).cuda()
    got, glse = K.kda_tree_attention(q.cuda(), kd, vd, table.cuda(), _i32(ctx).cuda(), tree_mask=mask,
                                     num_nodes=_dev(nodes), scale=scale, max_context=max_context, return_lse=True,
                                     device_status=status)
    assert status.item() == 0
    within(got, out, ob)
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(glse.cpu()) & (glse.cpu() < 0), empty)
    within(torch.where(empty, torch.zeros_like(lse), glse.cpu().to(lse.dtype)),
           torch.where(empty, torch.zeros_like(lse), lse), lb)
    assert bool((got.cpu()[empty] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,Hq,Hk", [(1, 4, 4), (1, 8, 1), (3, 6, 2), (4, 16, 4), (13, 10, 2), (40, 4, 1), (17, 16, 2)])
@pytest.mark.parametrize("room", [0, ROOM])
def test_tree_shapes(dtype, D, N, Hq, Hk, room):
    """Contexts around the tile sizes, an empty and a one-token one, one that is split."""
    _tree_case(N + Hq, [0, 1, 63, 64, 65, 128, 200, 700], N, Hq, Hk, D, 16, dtype, room=room)


@pytest.mark.parametrize("page,heads_first", [(1, False), (7, True), (8, False), (24, False), (64, True), (100, False),
                                              (4096, False)])
@pytest.mark.parametrize("N,G,room", [(2, 4, 0), (30, 8, 0), (5, 4, ROOM), (40, 8, ROOM)])
def test_tree_pages(page, heads_first, N, G, room):
    _tree_case(page, [130, 0, 900, 31], N, 2 * G, 2, 128, page, BF16, heads_first=heads_first, room=room)


@pytest.mark.parametrize("page", [8, 16, 24, 48, 128, 160, 512])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_pages_of_the_kernel_for_many_rows(page, heads_first, D):
    _tree_case(page, [513, 2, 127, 300, 0], 20, 12, 3, D, page, F16, heads_first=heads_first, room=ROOM)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N", [34, 48, 49, 100])
def test_tree_a_last_row_tile_by_itself(D, N):
    """Rows a little past 256, 384 and 768: the last pair of 128-row tiles full, half or hardly used."""
    _tree_case(N, [700, 5, 130], N, 8, 1, D, 16, BF16, room=ROOM)


@pytest.mark.parametrize("D,Hq,Hk,N", [(64, 4, 2, 3), (128, 8, 2, 1), (128, 12, 3, 8), (256, 16, 2, 1), (256, 2, 1, 20)])
@pytest.mark.parametrize("page", [3, 24, 64])
def test_tree_long_and_short_contexts_together(D, Hq, Hk, N, page):
    """Equal stretches of work that meet many requests, and a request that meets many stretches."""
    _tree_case(D + N, [6000, 0, 17, 2600, 1, 64, 3000, 127], N, Hq, Hk, D, page, BF16)


def test_tree_one_context_over_every_multiprocessor():
    _tree_case(5, [40000], 2, 4, 1, 128, 16, F16)


def test_tree_one_token_pages_of_a_long_context():
    """More pages in a stretch of work than are listed at a time."""
    _tree_case(6, [60000, 30000], 1, 4, 4, 64, 1, BF16)


def test_tree_many_requests_with_small_pages():
    """A CTA each, with more pages than are listed at a time."""
    _tree_case(7, [700 - 9 * i for i in range(40)], 1, 16, 8, 128, 2, BF16)


@pytest.mark.parametrize("rows", [40, 160])
def test_tree_few_items_in_many_parts(rows):
    """The joins of few and of many rows over many parts."""
    _tree_case(rows, [20000, 3], rows // 8, 8, 1, 128, 32, BF16)


def test_tree_cache_layouts_without_a_tensor_map():
    """Keys and values in one page, heads neither a row's nor a page's neighbours."""
    g = _gen(77)
    R, N, Hk, G, D, page = 2, 9, 3, 4, 64, 16
    table, total = _pages(g, [300, 64], page, room=ROOM)
    both = _rand(g, (total, page, Hk, 2, D), BF16)      # head stride 2 D
    q = _rand(g, (R, N, Hk * G, D), BF16)
    out, ob, _, _ = tree_reference(q, both[:, :, :, 0], both[:, :, :, 1], table, [291, 55])
    d = both.cuda()
    got = K.kda_tree_attention(q.cuda(), d[:, :, :, 0], d[:, :, :, 1], table.cuda(), _i32([291, 55]).cuda())
    within(got, out, ob)
    pages = _rand(g, (total, 2, page, Hk, D), BF16)     # a page's keys, then its values
    out, ob, _, _ = tree_reference(q, pages[:, 0], pages[:, 1], table, [291, 55])
    d = pages.cuda()
    got = K.kda_tree_attention(q.cuda(), d[:, 0], d[:, 1], table.cuda(), _i32([291, 55]).cuda())
    within(got, out, ob)


@pytest.mark.parametrize("N,form", [(1, "chain"), (5, "chain"), (64, "tree"), (65, "tree"), (130, "tree"),
                                    (256, "chain")])
@pytest.mark.parametrize("room", [0, ROOM])
def test_tree_node_counts(N, form, room):
    _tree_case(N, [77, 5], N, 2, 1, 64, 32, F16, form=form, room=room)


@pytest.mark.parametrize("N,room", [(9, 2048), (1, 0), (3, 0)])
def test_tree_many_requests(N, room):
    """More requests than one launch of the kernel for many rows takes (256), most of
    them short, some empty, some long enough to be cut; for few rows, more of them than
    the GPU runs at once, longest first."""
    ctx = [(i * 37) % 90 if i % 50 else 700 + i for i in range(300)]
    nodes = _i32([(i * 7) % (N + 1) for i in range(300)])
    _tree_case(50, ctx, N, 4, 2, 64, 16, BF16, nodes=nodes, room=room)


@pytest.mark.parametrize("G,room", [(2, 0), (12, ROOM)])
def test_tree_unused_nodes_and_nodes_outside_the_tree(G, room):
    """num_nodes below the call's, and nodes with parent -2 (their keys and values
    hold NaN): zero rows, no trace in the others."""
    g = _gen(3)
    parents = _random_parents(g, 4, 9)
    parents[0, 3], parents[2, 8], parents[3, 0] = -2, -2, -2
    for r in range(4):   # children of a node outside the tree hang behind the context
        for i in range(9):
            if parents[r, i] >= 0 and parents[r, int(parents[r, i])] == -2:
                parents[r, i] = -1
    for ctx in ([70, 0, 300, 5], [0, 0, 0, 0]):
        _tree_case(11, ctx, 9, 2 * G, 2, 128, 16, BF16, nodes=_i32([9, 0, 9, 4]), parents=parents, room=room)


def test_tree_values_that_only_some_rows_see_may_be_nan():
    """A node whose V holds NaN and infinity reaches its own descendants only."""
    g = _gen(5)
    for N, Hq, room in ((6, 4, 0), (24, 16, 0), (24, 16, ROOM), (70, 16, ROOM)):
        parents = torch.full((1, N), -1)
        parents[0, 2] = 1       # node 2 follows node 1, the rest follow the context
        table, total = _pages(g, [50 + N], 16, room=room)
        kc, vc = _rand(g, (total, 16, 2, 128), BF16), _rand(g, (total, 16, 2, 128), BF16)
        q = _rand(g, (1, N, Hq, 128), BF16)
        out, ob, _, _ = tree_reference(q, kc, vc, table, [50], sees=_sees(parents))
        p = 51                  # node 1's position
        vc[int(table[0, p // 16]), p % 16] = math.nan
        kc[int(table[0, p // 16]), p % 16, 0, 3] = math.inf
        got = K.kda_tree_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), _i32([50]).cuda(),
                                   tree_mask=K.tree_mask(parents).cuda()).cpu()
        assert bool(torch.isnan(got[0, 1:3]).all())
        rest = [i for i in range(N) if i not in (1, 2)]
        within(got[:, rest], out[:, rest], ob[:, rest])


def test_tree_large_scores_and_scales():
    """Scores of some hundreds (a softmax of one key), a negative and a zero scale."""
    _tree_case(21, [300, 64], 4, 4, 2, 128, 16, BF16, q_scale=30.0)
    _tree_case(22, [300, 64], 4, 4, 2, 128, 16, F16, scale=-0.1)
    _tree_case(23, [300, 64], 4, 4, 2, 64, 16, F16, scale=0.0)
    for dtype in (BF16, F16):
        _tree_case(24, [900, 64, 300], 12, 8, 2, 128, 16, dtype, q_scale=30.0, room=ROOM)


def test_tree_a_maximum_that_grows():
    """Scores that climb along the context: the running maximum has to move again and again."""
    for dtype, N, G, room in ((BF16, 3, 2, 0), (BF16, 20, 8, ROOM), (F16, 40, 8, ROOM), (F16, 6, 8, ROOM)):
        g = _gen(N)
        table, total = _pages(g, [1500], 16, room=room)
        kc, vc = _rand(g, (total, 16, 1, 128), dtype), _rand(g, (total, 16, 1, 128), dtype)
        q = _rand(g, (1, N, G, 128), dtype)
        q[..., 0] = 4.0
        for p in range(1500):
            kc[int(table[0, p // 16]), p % 16, 0, 0] = p / 10.0
        out, ob, lse, lb = tree_reference(q, kc, vc, table, [1500 - N], scale=0.3)
        got, glse = K.kda_tree_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), _i32([1500 - N]).cuda(),
                                         scale=0.3, return_lse=True)
        within(got, out, ob)
        within(glse, lse, lb)


@pytest.mark.parametrize("N,G,form", [(1, 8, "chain"), (16, 4, "tree"), (33, 8, "tree")])
def test_tree_long_context(N, G, form):
    _tree_case(31, [20011, 3], N, 2 * G, 2, 128, 64, BF16, poison=False, form=form)


def test_tree_max_context_changes_the_cut_only():
    _tree_case(32, [500, 20], 4, 8, 2, 128, 512, BF16, max_context=500)
    _tree_case(32, [500, 20], 4, 8, 2, 128, 512, BF16, max_context=100000)


def test_tree_strided_queries_and_outputs():
    g = _gen(33)
    table, total = _pages(g, [90, 41], 16)
    kc, vc = _rand(g, (total, 16, 2, 64), F16), _rand(g, (total, 16, 2, 64), F16)
    rows = _rand(g, (2, 3, 9, 64), F16)
    q = rows[:, :, 2:8]
    out, ob, _, _ = tree_reference(q, kc, vc, table, [87, 38])
    res = torch.full((2, 6, 8, 64), 5.0, dtype=F16, device="cuda")
    K.kda_tree_attention(rows.cuda()[:, :, 2:8], kc.cuda(), vc.cuda(), table.cuda(), _i32([87, 38]).cuda(),
                         out=res[:, ::2, 1:7])
    within(res[:, ::2, 1:7], out, ob)
    assert bool((res[:, 1::2] == 5.0).all()) and bool((res[:, :, 7] == 5.0).all())


@pytest.mark.parametrize("G,room", [(4, 0), (24, 0), (24, ROOM)])
def test_tree_reports_what_only_the_device_sees(G, room):
    g = _gen(34)
    table, total = _pages(g, [70, 70, 70], 16, spare=0, room=room)
    kc, vc = _rand(g, (total, 16, 1, 64), BF16).cuda(), _rand(g, (total, 16, 1, 64), BF16).cuda()
    q = _rand(g, (3, 2, G, 64), BF16).cuda()
    good = K.kda_tree_attention(q, kc, vc, table.cuda(), _i32([68, 60, 50]).cuda())

    def run(ctx, tab=table, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = K.kda_tree_attention(q, kc, vc, tab.cuda(), _i32(ctx).cuda(), device_status=status,
                                        return_lse=True, **kw)
        assert status.item() == 1
        return out, lse

    too_long = table.shape[1] * 16 - 1
    for ctx, kw in (([68, -1, 50], {}), ([68, too_long, 50], {}), ([68, 60, 50], dict(num_nodes=_i32([2, 3, 2]).cuda())),
                    ([68, 60, 50], dict(num_nodes=_i32([2, -1, 2]).cuda()))):
        out, lse = run(ctx, **kw)
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        assert bool((out[1] == 0).all()) and bool(torch.isinf(lse[1]).all())
    # a context past what the host was told
    out, _ = run([5, 60, 5], max_context=50)
    assert bool((out[1] == 0).all())
    # pages outside the cache read as zeros
    for bad in (-1, total):
        t2 = table.clone()
        t2[1, 1] = bad
        out, _ = run([68, 60, 50], t2)
        k0, v0 = kc.cpu().clone(), vc.cpu().clone()
        k0[int(table[1, 1])] = 0
        v0[int(table[1, 1])] = 0
        want, ob, _, _ = tree_reference(q.cpu(), k0, v0, table, [68, 60, 50])
        within(out, want, ob)


def test_tree_rows_past_2_to_31_elements():
    """A cache whose last pages start past 2^31 elements (of 16-bit keys)."""
    pages, page, D = 70000, 256, 128
    kc = torch.empty((pages, page, 1, D), dtype=BF16, device="cuda")
    vc = torch.empty((pages, page, 1, D), dtype=BF16, device="cuda")
    g = _gen(35)
    small_k, small_v = _rand(g, (2, page, 1, D), BF16), _rand(g, (2, page, 1, D), BF16)
    kc[pages - 2:], vc[pages - 2:] = small_k.cuda(), small_v.cuda()
    q = _rand(g, (1, 2, 4, D), BF16)
    table = _i32([[pages - 1, pages - 2]])
    out, ob, _, _ = tree_reference(q, small_k, small_v, _i32([[1, 0]]), [300])
    got = K.kda_tree_attention(q.cuda(), kc, vc, table.cuda(), _i32([300]).cuda())
    within(got, out, ob)
    # and the write into such a row
    freq, _ = K.rope_frequencies(128)
    k = _rand(g, (1, 1, D), BF16).cuda()
    K.kda_qk_norm_rope(k, k, _i32([0]).cuda(), freq, norm=False, v=k, k_cache=kc, v_cache=vc,
                       slots=torch.tensor([pages * page - 1], device="cuda"))
    assert torch.equal(kc[-1, -1], k[0]) and torch.equal(vc[-1, -1], k[0])


# ---------------------------------------------------------------- all of them
def _layer(x, w, st, qkv, pos, freq, slots, kc, vc, table, ctx):
    y = K.kda_short_conv(x, w, conv_state=st, norm_channels=256)
    q, _ = K.kda_qk_norm_rope(qkv[:, :4], qkv[:, 4:6], pos, freq, v=qkv[:, 6:], k_cache=kc, v_cache=vc, slots=slots)
    return y, K.kda_tree_attention(q.view(2, 3, 4, 128), kc, vc, table, ctx)


def _layer_inputs():
    g = _gen(40)
    x, w = _rand(g, (2, 3, 384), BF16).cuda(), _rand(g, (384, 4), torch.float32).cuda()
    st = _rand(g, (2, 3, 384), BF16).cuda()
    qkv = _rand(g, (6, 8, 128), BF16).cuda()
    freq, _ = K.rope_frequencies(128)
    table = _i32([list(range(0, 40)), list(range(40, 80))]).cuda()
    ctx = _i32([600, 17]).cuda()
    pos = _i32([600, 601, 602, 17, 18, 19]).cuda()
    slots = torch.tensor([600, 601, 602, 640 + 17, 640 + 18, 640 + 19], device="cuda")
    kc, vc = _rand(g, (80, 16, 2, 128), BF16).cuda(), _rand(g, (80, 16, 2, 128), BF16).cuda()
    return x, w, st, qkv, pos, freq, slots, kc, vc, table, ctx


def test_ops_on_another_stream_and_in_a_graph():
    a = _layer_inputs()
    st0 = a[2].clone()
    y, o = _layer(*a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a[2].copy_(st0)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, o2 = _layer(*a)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(o, o2)
    a[2].copy_(st0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, o3 = _layer(*a)
    for _ in range(2):
        a[2].copy_(st0)
        y3.zero_()
        o3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y3) and torch.equal(o, o3)


def test_ops_give_the_same_bits_again():
    a = _layer_inputs()
    st0 = a[2].clone()
    first = None
    for _ in range(5):
        a[2].copy_(st0)
        r = _layer(*a)
        first = first or r
        assert torch.equal(r[0], first[0]) and torch.equal(r[1], first[1])

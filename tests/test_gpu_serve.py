"""Chunk attention, the residual stream's norm, pool copies and the commit of verified
trees' cache rows on the GPU against their 64-bit forms."""
import math

import pytest
import torch

import kda_chunked_prefill_02_gb300 as K
from ops_test_util import within
from serve_test_util import chunk_reference, residual_reference

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- chunk attention
def _chunk_inputs(seed, ctx, new, Hq, Hk, D, page, dtype, room=0, extra_pages=2):
    """q, caches, table, contexts and cu_seqlens on the host: every request its own pages."""
    g = _gen(seed)
    need = [(c + n + page - 1) // page for c, n in zip(ctx, new)]
    table = torch.zeros((len(ctx), max(max(need), room // page, 1)), dtype=torch.int32)
    order, at = torch.randperm(sum(need) + extra_pages, generator=g).to(torch.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    pages = sum(need) + extra_pages
    kc, vc = _rand(g, (pages, page, Hk, D), dtype), _rand(g, (pages, page, Hk, D), dtype)
    return (_rand(g, (sum(new), Hq, D), dtype, 1.5), kc, vc, table, _i32(ctx),
            _i32([0] + new).cumsum(0).to(torch.int32))


def _check(q, kc, vc, table, ctx, cu, got, lse, **kw):
    new = (cu[1:] - cu[:-1]).tolist()
    out, ob, want, lb = chunk_reference(q, kc, vc, table, ctx, new, **kw)
    within(got, out, ob)
    if lse is not None:
        lse = lse.cpu()
        seen = torch.isfinite(want)
        assert torch.equal(torch.isfinite(lse), seen)
        within(torch.where(seen, lse, 0), torch.where(seen, want, 0), torch.where(seen, lb, 0))


# tokens a page table has room for: enough for the tensor-core kernel, whatever the lengths
ROOM = 300000


def _kernel(q, kc, table, **kw):
    return K.chunk_attention_schedule(q, kc, table, packed=q.dim() == 3, **kw)["kernel"]


def _chunk_case(seed, ctx, new, Hq, Hk, D, page, dtype, *, scale=None, room=0, max_context=None, kernel=None):
    q, kc, vc, table, lens, cu = _chunk_inputs(seed, ctx, new, Hq, Hk, D, page, dtype, room)
    status = _status()
    if kernel:
        assert _kernel(q, kc, table, scale=scale, max_context=max_context) == kernel
    got, lse = K.kda_chunk_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), cu_seqlens=cu.cuda(),
                                     scale=scale, max_context=max_context, return_lse=True, device_status=status)
    assert status.item() == 0
    _check(q, kc, vc, table, lens, cu, got, lse, scale=scale)


RAGGED = ([0, 700, 1, 64, 63, 127, 200, 5], [1, 0, 5, 33, 130, 64, 1, 128])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("Hq,Hk,page", [(2, 2, 16), (8, 2, 64), (16, 1, 128), (10, 2, 24), (3, 1, 5), (6, 2, 100)])
def test_chunk_ragged(dtype, D, Hq, Hk, page, room):
    _chunk_case(1, *RAGGED, Hq, Hk, D, page, dtype, room=room, kernel="tensor" if room and page % 8 == 0 else None)


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("Hq,Hk", [(7, 1), (12, 1), (20, 1), (48, 1), (100, 1), (128, 1), (200, 1), (256, 1), (300, 1)])
def test_chunk_query_heads_of_a_key_head(Hq, Hk, room):
    """Row tiles that are not full, and more query heads than a row tile has rows."""
    _chunk_case(2, [130, 0, 9], [3, 40, 17], Hq, Hk, 64, 16, BF16, room=room,
                kernel="tensor" if room and Hq <= 128 else None)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_chunk_of_one_request(dtype, tokens, room):
    """Last row tiles of every kind, key tiles that end inside and at the tokens' own."""
    for ctx in (0, 1, 95, 96, 97, 127, 128, 1000):
        _chunk_case(3, [ctx], [tokens], 8, 2, 128, 64, dtype, room=room, kernel="tensor" if room else None)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("tokens", [128, 129, 255, 256, 257, 600])
def test_chunk_row_tiles_that_see_different_key_tiles(D, tokens):
    """One query head a key head: the first of two row tiles ends before the last key tile."""
    for ctx in (0, 1, 64, 127):
        _chunk_case(21, [ctx, 5], [tokens, 140], 2, 2, D, 16, BF16, room=ROOM, kernel="tensor")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx", [0, 6000])
def test_chunk_long(D, ctx):
    """Many blocks of rows, many tiles a block."""
    _chunk_case(4, [ctx, 100], [1500, 300], 4, 1, D, 16, BF16)


def test_chunk_many_requests():
    """More requests than a warp looks at in one go, single tokens between longer pieces."""
    ctx = [(i * 37) % 300 if i % 50 else 900 + i for i in range(400)]
    new = [1 if i % 7 else (i * 13) % 90 for i in range(400)]
    _chunk_case(5, ctx, new, 4, 2, 64, 16, BF16, kernel="rows")
    _chunk_case(5, ctx, new, 8, 2, 128, 16, BF16, room=ROOM, kernel="tensor")
    _chunk_case(6, ctx[:70], new[:70], 8, 2, 128, 16, F16, max_context=max(ctx))


@pytest.mark.parametrize("kernel", ["rows", "tensor"])
def test_chunk_thousands_of_requests(kernel):
    """Runs of requests without tokens among single tokens and short pieces; a decrease of
    cu_seqlens is reported wherever it is."""
    R = 5000
    new = [0 if i % 9 < 6 else 1 + (i % 5) * (i % 70 == 7) for i in range(R)]
    ctx = [(i * 7) % 30 for i in range(R)]
    D = 64 if kernel == "rows" else 128
    q, kc, vc, table, lens, cu = _chunk_inputs(27, ctx, new, 2, 1, D, 16, BF16, 0 if kernel == "rows" else 20000)
    dev = [t.cuda() for t in (q, kc, vc, table, lens)]
    assert _kernel(q, kc, table) == kernel
    status = _status()
    got = K.kda_chunk_attention(*dev, cu_seqlens=cu.cuda(), device_status=status)
    assert status.item() == 0
    _check(q, kc, vc, table, lens, cu, got, None)
    for at in (1, 31, 32, 33, 2500, 4999):
        bad = cu.clone()
        bad[at] = -1 if at % 2 else int(cu[-1]) + 1
        status.zero_()
        K.kda_chunk_attention(*dev, cu_seqlens=bad.cuda(), device_status=status)
        assert status.item() == 1


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("T", [1, 3, 40, 140])
def test_chunk_padded(T, room):
    """[R, T, Hq, D]: as the packed form of equal lengths."""
    ctx = [0, 77, 300]
    q, kc, vc, table, lens, cu = _chunk_inputs(7, ctx, [T] * 3, 8, 2, 128, 16, BF16, room)
    got, lse = K.kda_chunk_attention(q.view(3, T, 8, 128).cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(),
                                     return_lse=True)
    assert got.shape == (3, T, 8, 128) and lse.shape == (3, T, 8)
    _check(q, kc, vc, table, lens, cu, got.flatten(0, 1), lse.flatten(0, 1))


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("scale", [1.0, 0.01, 0.0, -0.3, 1e-38])
def test_chunk_scales(scale, room):
    """Scales that are not above zero, or whose reciprocal is no fp32 number, take the kernel for few rows."""
    _chunk_case(8, [100, 0], [30, 200], 4, 1, 64, 16, BF16, scale=scale, room=room,
                kernel=("tensor" if scale > 1e-30 else "rows") if room else None)


@pytest.mark.parametrize("room", [0, ROOM])
def test_chunk_strides(room):
    """q as heads of a fused projection, results into a wider buffer, caches with the heads
    before the rows, with keys and values in one tensor, and with rows that belong to no map."""
    ctx, new = [50, 0, 260], [70, 5, 129]
    q, kc, vc, table, lens, cu = _chunk_inputs(9, ctx, new, 8, 2, 128, 16, BF16, room)
    T = sum(new)
    wide = torch.zeros(T, 14, 128, dtype=BF16, device="cuda")
    wide[:, 3:11] = q.cuda()
    dev = dict(cu_seqlens=cu.cuda())
    tab, ln = table.cuda(), lens.cuda()
    heads_first = [c.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) for c in (kc, vc)]
    together = torch.stack([kc, vc], 2).cuda()
    spread = torch.zeros(kc.shape[0], 16, 2, 2, 136, dtype=BF16, device="cuda")
    spread[..., 0, :128], spread[..., 1, :128] = kc.cuda(), vc.cuda()
    for k, v in (heads_first, (together[:, :, 0], together[:, :, 1]), (spread[..., 0, :128], spread[..., 1, :128])):
        res = torch.full((T, 10, 128), 7.0, dtype=BF16, device="cuda")
        got = K.kda_chunk_attention(wide[:, 3:11], k, v, tab, ln, out=res[:, 1:9], **dev)
        _check(q, kc, vc, table, lens, cu, got, None)
        assert bool((res[:, 0] == 7).all()) and bool((res[:, 9] == 7).all())
        # results that start on 16 bytes, not on 32
        odd = torch.full((T * 1032 + 8,), 7.0, dtype=BF16, device="cuda")[8:].view(T, 1032)[:, :1024].view(T, 8, 128)
        got = K.kda_chunk_attention(wide[:, 3:11], k, v, tab, ln, out=odd, **dev)
        _check(q, kc, vc, table, lens, cu, got, None)


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx,new", [([300], [4]), ([0, 90, 4000], [300, 1, 37])])
def test_chunk_results_over_the_queries(D, ctx, new, room):
    q, kc, vc, table, lens, cu = _chunk_inputs(10, ctx, new, 8, 2, D, 16, BF16, room)
    qd = q.cuda()
    got = K.kda_chunk_attention(qd, kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), cu_seqlens=cu.cuda(), out=qd)
    assert got is qd
    _check(q, kc, vc, table, lens, cu, got, None)


@pytest.mark.parametrize("room", [0, ROOM])
def test_chunk_rows_behind_the_last_request_are_left(room):
    """A batch padded to a fixed number of rows, whatever the padding holds."""
    ctx, new = [20, 3], [33, 70]
    q, kc, vc, table, lens, cu = _chunk_inputs(11, ctx, new, 8, 2, 128, 16, BF16, room)
    T = sum(new)
    qd = torch.full((T + 100, 8, 128), math.nan, dtype=BF16, device="cuda")
    qd[:T] = q.cuda()
    res = torch.full_like(qd, 7.0)
    status = _status()
    K.kda_chunk_attention(qd, kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), cu_seqlens=cu.cuda(), out=res,
                          device_status=status)
    assert status.item() == 0
    _check(q, kc, vc, table, lens, cu, res[:T], None)
    assert bool((res[T:] == 7).all())


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("D,Hq,Hk,page", [(128, 8, 2, 16), (64, 2, 2, 64), (256, 4, 1, 24), (128, 4, 2, 10)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_chunk_what_a_row_does_not_see(D, Hq, Hk, page, what, dtype, room):
    """Unused pages, rows behind a request's end, and the keys of its last tokens: only the
    rows that see a token feel it.  Values that are not finite reach those."""
    ctx, new = [70, 0, 129], [90, 40, 3]
    q, kc, vc, table, lens, cu = _chunk_inputs(12, ctx, new, Hq, Hk, D, page, dtype, room)
    clean_k, clean_v = kc.clone(), vc.clone()
    used = torch.zeros(kc.shape[0], page, dtype=torch.bool)
    for r in range(3):
        at = torch.arange(ctx[r] + new[r])
        used[table[r].long()[at // page], at % page] = True
    kc[~used], vc[~used] = what, what
    clean_k[~used], clean_v[~used] = 0, 0

    def place(r, p):
        return int(table[r, p // page]), p % page

    hidden = []          # (request, new token): its own row and those behind it see it
    for r, i in ((0, 41), (1, 17), (1, 38), (2, 2)):
        a, b = place(r, ctx[r] + i)
        vc[a, b, Hk - 1, 3::5] = what
        clean_v[a, b, Hk - 1, 3::5] = 0
        hidden.append((r, i))
    got = K.kda_chunk_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), cu_seqlens=cu.cuda()).cpu()
    out, ob, _, _ = chunk_reference(q, clean_k, clean_v, table, lens, new)
    hit = torch.zeros(q.shape, dtype=torch.bool)
    for r, i in hidden:
        hit[int(cu[r]) + i:int(cu[r + 1]), (Hk - 1) * (Hq // Hk):, 3::5] = True
    assert bool((torch.isnan(got[hit]) if math.isnan(what) else got[hit] == what).all())
    within(torch.where(hit, 0, got), torch.where(hit, 0, out), torch.where(hit, 1.0, ob))


@pytest.mark.parametrize("room", [0, ROOM])
def test_chunk_keys_that_are_not_finite(room):
    """A key that is NaN makes NaN of the rows that see it, and of no other."""
    ctx, new = [10], [200]
    q, kc, vc, table, lens, cu = _chunk_inputs(13, ctx, new, 4, 1, 128, 16, BF16, room)
    out, ob, _, _ = chunk_reference(q, kc, vc, table, lens, new)
    p = 10 + 150
    kc[int(table[0, p // 16]), p % 16, 0, 7] = math.nan
    got = K.kda_chunk_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), cu_seqlens=cu.cuda()).cpu()
    assert bool(torch.isnan(got[150:]).all())
    within(got[:150], out[:150], ob[:150])


@pytest.mark.parametrize("room", [0, ROOM])
def test_chunk_reports_what_only_the_device_sees(room):
    ctx, new = [20, 30, 40, 50], [9, 70, 1, 30]
    q, kc, vc, table, lens, cu = _chunk_inputs(14, ctx, new, 8, 2, 128, 16, BF16, room)
    out, ob, lse_ref, _ = chunk_reference(q, kc, vc, table, lens, new)
    dev = [t.cuda() for t in (q, kc, vc, table)]

    def run(lens, cu, table=None, **kw):
        status = _status()
        res = torch.full(q.shape, 7.0, dtype=BF16, device="cuda")
        got, lse = K.kda_chunk_attention(dev[0], dev[1], dev[2], dev[3] if table is None else table.cuda(), lens.cuda(),
                                         cu_seqlens=cu.cuda(), device_status=status, out=res, return_lse=True, **kw)
        return got.cpu(), lse.cpu(), status.item()

    a, b = int(cu[1]), int(cu[2])
    for bad, kw in ((-1, {}), (table.shape[1] * 16 - 69, {}), (1 << 30, {}), ((1 << 31) - 1, {}), (45, dict(max_context=44))):
        ln = lens.clone()
        ln[1] = bad
        if kw:
            ln[3] = 44
        got, lse, st = run(ln, cu, **kw)
        assert st == 1
        assert bool((got[a:b] == 0).all()) and bool((lse[a:b] == -math.inf).all())
        within(got[:a], out[:a], ob[:a])
        within(got[b:b + 1], out[b:b + 1], ob[b:b + 1])
    # bounds that do not start at 0, decrease, or pass the rows
    for bad in ([0, 9, 200, 80, 110], [0, 9, 5, 80, 110], [0, 9, -4, 80, 110], [3, 9, 79, 80, 110]):
        got, _, st = run(lens, _i32(bad))
        assert st == 1
    # the same rows over and over: no more work than the call's rows
    again = _i32([0, int(cu[-1])] * 2 + [0])
    assert run(lens, again)[2] == 1
    for good in ([0, 9, 9, 9, 9], [0, 0, 0, 0, 0], [0, 9, 79, 80, 100]):
        assert run(lens, _i32(good))[2] == 0
    # pages outside the pool read as zeros
    t2 = table.clone()
    t2[1, 2], t2[1, 3] = kc.shape[0], -5
    zk, zv = torch.cat([kc, torch.zeros_like(kc[:1])]), torch.cat([vc, torch.zeros_like(vc[:1])])
    t3 = t2.clone()
    t3[1, 2] = t3[1, 3] = kc.shape[0]
    got, _, st = run(lens, cu, table=t2)
    assert st == 1
    o3, b3, _, _ = chunk_reference(q, zk, zv, t3, lens, new)
    within(got, o3, b3)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("gap", [13.0, 17.5, 20.0])
@pytest.mark.parametrize("n,R", [(1, 1), (30, 1), (30, 200)])
def test_chunk_weight_in_many_keys_far_below_the_largest(dtype, gap, n, R):
    """One key whose score is `gap` above all others' and whose value is 0, before 150000 keys
    with values near 1: the result is the many keys' share, 150000 e^-gap of the whole.  A
    weight's rounding to fp16 is off by its unit, or where it is smaller by half of 2^-24 at
    the kernels' scales (2^11 at least).  As many equal requests as make a CTA take a context
    whole, and one alone."""
    L, page = 150000, 16
    q, kc, vc, table, lens, cu = _chunk_inputs(15, [L], [n], 2, 1, 64, page, dtype)
    g = _gen(16)
    q[:], kc[:] = 0, 0
    q[..., 0] = 1.0
    vc.copy_(1 + _rand(g, vc.shape, F32, 0.1))
    at = int(table[0, 77])
    kc[at, 5, 0, 0], vc[at, 5] = gap, 0
    out, ob, lse, lb = chunk_reference(q, kc, vc, table, lens, [n], scale=1.0)
    if dtype == F16:
        ob = ob + (L + n) * 2.0 ** -25 * 2.0 ** -11 * vc.abs().max().double()
    got, glse = K.kda_chunk_attention(q[None].expand(R, n, 2, 64).contiguous().cuda(), kc.cuda(), vc.cuda(),
                                      table.expand(R, -1).contiguous().cuda(), lens.expand(R).contiguous().cuda(),
                                      scale=1.0, return_lse=True)
    for r in (0, R // 2, R - 1):
        within(got[r], out, ob)
        within(glse[r], lse, lb)


@pytest.mark.parametrize("room", [0, ROOM])
def test_chunk_offsets_past_32_bits(room):
    """A cache of more than 2^32 bytes: the pages at its end."""
    pages, page, Hk, D = 70000, 64, 4, 128
    kc = torch.zeros(pages, page, Hk, D, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() > 1 << 31
    ctx, new = [150, 10], [40, 3]
    q, ks, vs, table, lens, cu = _chunk_inputs(17, ctx, new, 8, Hk, D, page, BF16, room)
    far = pages - ks.shape[0]
    kc[far:], vc[far:] = ks.cuda(), vs.cuda()
    got = K.kda_chunk_attention(q.cuda(), kc, vc, (table + far).cuda(), lens.cuda(), cu_seqlens=cu.cuda())
    _check(q, ks, vs, table, lens, cu, got, None)


def test_chunk_in_pieces_and_as_drafts():
    """A prompt in pieces, and its tokens as chains of drafts: the same rows within one
    rounding of the weights and the results on either side (2^-7 of the values' size)."""
    n = 333
    q, kc, vc, table, lens, cu = _chunk_inputs(18, [0], [n], 8, 2, 128, 16, BF16)
    dev = [t.cuda() for t in (kc, vc, table)]
    whole = K.kda_chunk_attention(q.cuda(), *dev, lens.cuda(), cu_seqlens=cu.cuda())
    out, ob, _, _ = chunk_reference(q, kc, vc, table, lens, [n])
    at = 0
    for piece in (1, 2, 61, 64, 200, 5):
        part = K.kda_chunk_attention(q[at:at + piece].cuda(), *dev, _i32([at]).cuda(), cu_seqlens=_i32([0, piece]).cuda())
        within(part, out[at:at + piece], ob[at:at + piece])
        at += piece
    within(whole, out, ob)
    drafts = K.kda_tree_attention(q[300:333][None].cuda(), *dev, _i32([300]).cuda())
    within(drafts[0], out[300:], ob[300:])


@pytest.mark.parametrize("room", [8192, ROOM])
def test_chunk_repeats_and_graphs(room):
    """The same bits each time, on other streams, and from a captured call whose lengths are
    those of the replay."""
    ctx, new = [500, 0, 3000, 77], [30, 250, 1, 129]
    q, kc, vc, table, lens, cu = _chunk_inputs(19, ctx, new, 8, 2, 128, 16, BF16, room=room)
    dev = [t.cuda() for t in (q, kc, vc, table, lens)]
    cud = cu.cuda()
    first = K.kda_chunk_attention(*dev, cu_seqlens=cud)
    for _ in range(5):
        assert torch.equal(K.kda_chunk_attention(*dev, cu_seqlens=cud), first)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    res = [K.kda_chunk_attention(*dev, cu_seqlens=cud, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, first) for x in res)

    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(first)
    ln, c2 = torch.zeros_like(dev[4]), torch.zeros_like(cud)
    with torch.cuda.graph(graph):
        K.kda_chunk_attention(*dev[:4], ln, cu_seqlens=c2, out=out)
    ln.copy_(dev[4])
    c2.copy_(cud)
    graph.replay()
    assert torch.equal(out, first)
    other = _i32([0, 100, 101, 220, 410]).cuda()
    ln.copy_(_i32([10, 2000, 0, 300]))
    c2.copy_(other)
    graph.replay()
    assert torch.equal(out, K.kda_chunk_attention(*dev[:4], _i32([10, 2000, 0, 300]).cuda(), cu_seqlens=other))


KDA_ERR_TIMEOUT = 4


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx,new", [([3000, 0, 900, 17], [24, 1, 7, 30]), ([20000, 5, 300, 700] * 8, [300, 64, 1, 500] * 8)])
def test_chunk_wait_that_runs_out_is_reported_and_the_context_survives(D, ctx, new):
    """The first wait of the softmax warps is for a barrier that nothing arrives on, so that it
    runs out with copies and products in flight.  The call returns and says so, and the next
    one on the same stream and workspace gives the usual bits."""
    pages = 4000   # the requests share them
    kc = torch.randn(pages, 16, 2, D, device="cuda").to(BF16)
    vc = torch.randn_like(kc)
    g = _gen(23)
    table = torch.randint(0, pages, (len(ctx), ROOM // 16), generator=g).to(torch.int32).cuda()
    q, lens = _rand(g, (sum(new), 8, D), BF16).cuda(), _i32(ctx).cuda()
    cu = _i32([0] + new).cumsum(0).to(torch.int32).cuda()
    assert _kernel(q, kc, table) == "tensor"
    status = _status()
    usual = K.kda_chunk_attention(q, kc, vc, table, lens, cu_seqlens=cu, device_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for limit in (2000, 200000):
        with K.overrides(wait_limit_ns=limit, timeout_probe=True):
            K.kda_chunk_attention(q, kc, vc, table, lens, cu_seqlens=cu, device_status=status)
        torch.cuda.synchronize()            # returns: no hang, no fault
        assert status.item() == KDA_ERR_TIMEOUT
        status.zero_()
        again = K.kda_chunk_attention(q, kc, vc, table, lens, cu_seqlens=cu, device_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0 and torch.equal(again, usual)


def test_chunk_waits_that_last_as_long_as_an_item_do_not_run_out():
    """Items of 8192 key tiles take a CTA some 14 ms; the bound of a wait here is 1 ms beside
    what the contexts themselves may take."""
    g = _gen(24)
    R, pages = 38, 600   # the requests share their pages
    kc, vc = (torch.randn(pages, 64, 4, 128, device="cuda").to(BF16) for _ in range(2))
    table = torch.randint(0, pages, (R, (1 << 14) + 1), generator=g).to(torch.int32).cuda()
    q, lens = _rand(g, (R, 32, 32, 128), BF16).cuda(), torch.full((R,), 1 << 20, dtype=torch.int32).cuda()
    status = _status()
    usual = K.kda_chunk_attention(q, kc, vc, table, lens)
    with K.overrides(wait_limit_ns=1000000):
        got = K.kda_chunk_attention(q, kc, vc, table, lens, device_status=status)
    assert status.item() == 0 and torch.equal(got, usual)


def test_one_token_as_a_transposed_column():
    """The row of a transposed column has strides (1, 1): what a matrix times a column leaves
    behind.  Every operator takes it as the contiguous row that it is."""
    g = _gen(25)

    def row(n):
        r = _rand(g, (n, 1), BF16).cuda().t()
        assert r.stride() == (1, 1) and r.is_contiguous()
        return r

    for room in (0, ROOM):
        q, kc, vc, table, lens, cu = _chunk_inputs(26, [200], [1], 4, 2, 128, 16, BF16, room)
        dev = [t.cuda() for t in (kc, vc, table, lens)]
        qd = row(512).as_strided((1, 4, 128), (1, 128, 1))
        want = K.kda_chunk_attention(qd.contiguous().clone(), *dev, cu_seqlens=cu.cuda())
        assert torch.equal(K.kda_chunk_attention(qd, *dev, cu_seqlens=cu.cuda()), want)
    x, y = row(384), row(384)
    a, b = K.kda_residual_norm(x, y), K.kda_residual_norm(x.clone().view(1, 384), y.clone().view(1, 384))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    pool = torch.arange(2 * 64, dtype=F32, device="cuda").view(2, 1, 64).as_strided((2, 1, 64), (64, 1, 1))
    K.kda_pool_copy(pool, _i32([0]).cuda(), _i32([1]).cuda())
    assert torch.equal(pool[1], pool[0])


# ---------------------------------------------------------------- the residual stream's norm
def _norm_case(seed, T, E, dtype, xdtype, *, post=False, gate=None, sigmoid=False, wdtype=F32, scale=1.0, alpha=0.7,
               weight=True, **kw):
    g = _gen(seed)
    x, y = _rand(g, (T, E), xdtype, 2.0 * scale), _rand(g, (T, E), dtype, scale)
    w = (1 + _rand(g, (E,), F32, 0.2)).to(wdtype) if weight else None
    pw = (1 + _rand(g, (E,), F32, 0.2)).to(wdtype) if post and weight else None
    gt = None if gate is None else _rand(g, (E,) if gate == "one" else (T, E), dtype, 2.0)
    h, hb, nx, xb = residual_reference(x, y, weight=w, post_norm=post, post_weight=pw, gate=gt, gate_sigmoid=sigmoid,
                                       alpha=alpha)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    gh, gx = K.kda_residual_norm(x.cuda(), y.cuda(), weight=dev(w), post_norm=post, post_weight=dev(pw), gate=dev(gt),
                                 gate_sigmoid=sigmoid, alpha=alpha, **kw)
    assert gh.dtype == dtype and gx.dtype == xdtype
    within(gh, h, hb)
    within(gx, nx, xb)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("E", [8, 64, 504, 512, 520, 1024, 1288, 2048, 4096, 8200, 16384])
def test_norm_widths(dtype, E):
    _norm_case(1, 5, E, dtype, dtype)
    _norm_case(2, 9, E, dtype, F32, post=True, gate="all", sigmoid=True, wdtype=dtype)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 127, 1000])
@pytest.mark.parametrize("E", [256, 1288])
def test_norm_tokens(T, E):
    _norm_case(3, T, E, BF16, BF16, post=True, gate="all")


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate,sigmoid", [(None, False), ("one", False), ("one", True), ("all", False), ("all", True)])
@pytest.mark.parametrize("xdtype", [BF16, F32])
@pytest.mark.parametrize("weight", [False, True])
def test_norm_forms(post, gate, sigmoid, xdtype, weight):
    _norm_case(4, 37, 1032, BF16, xdtype, post=post, gate=gate, sigmoid=sigmoid, weight=weight)


def test_norm_sizes_of_values():
    _norm_case(5, 6, 640, BF16, BF16, scale=1e8, post=True)
    _norm_case(6, 6, 640, BF16, F32, scale=1e-4)
    _norm_case(7, 6, 640, BF16, BF16, scale=0.0, norm_eps=1e-6)
    _norm_case(8, 6, 640, BF16, BF16, alpha=0.0)
    _norm_case(9, 6, 640, BF16, BF16, alpha=-3.0)


def test_norm_alone_and_sum_alone():
    g = _gen(10)
    x, y, w = _rand(g, (3, 7, 256), BF16), _rand(g, (3, 7, 256), BF16), _rand(g, (256,), F32)
    h, hb, _, _ = residual_reference(x, None, weight=w)
    xd = x.cuda()
    got, same = K.kda_residual_norm(xd, weight=w.cuda())
    assert same is xd
    within(got, h, hb)
    x32 = x.float() * 1.001
    h, hb, _, _ = residual_reference(x32, None, weight=w, dtype=F16)
    got, _ = K.kda_residual_norm(x32.cuda(), weight=w.cuda(), out=torch.empty(3, 7, 256, dtype=F16, device="cuda"))
    within(got, h, hb)
    none, nx = K.kda_residual_norm(xd, y.cuda(), norm=False, alpha=0.5)
    assert none is None
    _, _, want, xb = residual_reference(x, y, alpha=0.5)
    within(nx, want, xb)


def test_norm_strides_and_results_over_the_inputs():
    g = _gen(11)
    x, y, w = _rand(g, (33, 520), BF16), _rand(g, (33, 520), BF16), _rand(g, (520,), F32)
    h, hb, nx, xb = residual_reference(x, y, weight=w)
    wide_x, wide_y = torch.full((33, 1040), 7.0, dtype=BF16, device="cuda"), torch.full((33, 528), 7.0, dtype=BF16, device="cuda")
    wide_x[:, 520:], wide_y[:, 8:] = x.cuda(), y.cuda()
    gh, gx = K.kda_residual_norm(wide_x[:, 520:], wide_y[:, 8:], weight=w.cuda(), out=wide_y[:, 8:], x_out=wide_x[:, 520:])
    within(gh, h, hb)
    within(gx, nx, xb)
    assert gh.data_ptr() == wide_y[:, 8:].data_ptr() and gx.data_ptr() == wide_x[:, 520:].data_ptr()
    assert bool((wide_x[:, :520] == 7).all()) and bool((wide_y[:, :8] == 7).all())
    # one gate for all tokens, as an expanded row
    gate = _rand(g, (520,), BF16)
    a = K.kda_residual_norm(x.cuda(), y.cuda(), gate=gate.cuda())
    b = K.kda_residual_norm(x.cuda(), y.cuda(), gate=gate.cuda().expand(33, 520))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_rows_that_are_not_finite_stay_by_themselves():
    g = _gen(12)
    x, y = _rand(g, (9, 256), BF16), _rand(g, (9, 256), BF16)
    h, hb, nx, xb = residual_reference(x, y, post_norm=True)
    y[4, 17] = math.inf
    gh, gx = K.kda_residual_norm(x.cuda(), y.cuda(), post_norm=True)
    keep = torch.arange(9) != 4
    within(gh[keep.cuda()], h[keep], hb[keep])
    assert bool(torch.isnan(gh[4]).any())


def test_norm_no_tokens():
    e = torch.empty(0, 256, dtype=BF16, device="cuda")
    h, x = K.kda_residual_norm(e, e)
    assert h.shape == (0, 256) and x.shape == (0, 256)


# ---------------------------------------------------------------- pool copies
@pytest.mark.parametrize("dtype", [BF16, F32, torch.uint8, torch.int64])
def test_copy_entries(dtype):
    g = _gen(20)
    shapes = [(11, 16, 2, 128), (11, 3, 384), (11, 4, 128, 128), (11, 16), (11, 1, 1, 16), (11, 64, 8, 16, 16)]
    pools = [torch.randint(0, 100, s, generator=g).to(dtype) for s in shapes]
    src, dst = [0, 3, 3, -1, 5, 6], [1, 2, 10, 4, -7, 6]
    want = [p.clone() for p in pools]
    for w, p in zip(want, pools):
        for a, b in ((0, 1), (3, 2), (3, 10)):
            w[b] = p[a]
    dev = [p.cuda() for p in pools]
    status = _status()
    assert K.kda_pool_copy(dev, _i32(src).cuda(), _i32(dst).cuda(), device_status=status) is None
    assert status.item() == 0
    assert all(torch.equal(d.cpu(), w) for d, w in zip(dev, want))
    # a single pool, and its first rows alone
    one = pools[0].cuda()
    rows = [16, 5, 0, 3, 1, 16]
    want = pools[0].clone()
    for (a, b), n in zip(((0, 1), (3, 2), (3, 10)), rows):
        want[b, :n] = pools[0][a, :n]
    K.kda_pool_copy(one, _i32(src).cuda(), _i32(dst).cuda(), rows=_i32(rows).cuda())
    assert torch.equal(one.cpu(), want)


def test_copy_strides():
    """Heads before rows, both halves of a joint cache, and entries of a wider buffer."""
    g = _gen(21)
    base = _rand(g, (7, 4, 16, 64), BF16).cuda()
    joint = _rand(g, (7, 16, 2, 3, 64), BF16).cuda()
    wide = _rand(g, (7, 10, 80), BF16).cuda()
    pools = [base.permute(0, 2, 1, 3), joint[:, :, 0], wide[:, :, 8:72]]
    before = [t.clone() for t in (base, joint, wide)]
    rows = [9, 10]
    K.kda_pool_copy(pools, _i32([1, 4]).cuda(), _i32([6, 0]).cuda(), rows=_i32(rows).cuda())
    want = [t.clone() for t in before]
    views = [want[0].permute(0, 2, 1, 3), want[1][:, :, 0], want[2][:, :, 8:72]]
    for v, b in zip(views, (before[0].permute(0, 2, 1, 3), before[1][:, :, 0], before[2][:, :, 8:72])):
        for (s, d), n in zip(((1, 6), (4, 0)), rows):
            v[d, :n] = b[s, :n]
    for got, w in zip((base, joint, wide), want):
        assert torch.equal(got, w)


def test_copy_many_pools_and_large_entries():
    """More pools than a launch takes, entries of several slices with an odd end."""
    g = _gen(22)
    pools = [_rand(g, (5, 3, 8 * (40 + i)), BF16).cuda() for i in range(100)]
    want = [p.clone() for p in pools]
    for w in want:
        w[4] = w[1]
        w[0] = w[2]
    K.kda_pool_copy(pools, _i32([1, 2]).cuda(), _i32([4, 0]).cuda())
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    big = torch.arange(3 * 70001 * 8, dtype=torch.int32, device="cuda").view(3, 70001, 8)
    want = big.clone()
    want[2, :70000] = want[0, :70000]
    K.kda_pool_copy(big, _i32([0]).cuda(), _i32([2]).cuda(), rows=_i32([70000]).cuda())
    assert torch.equal(big, want)


def test_copy_reports_what_only_the_device_sees():
    p = torch.arange(5 * 4 * 8, dtype=torch.int32, device="cuda").view(5, 4, 8)
    want = p.clone()
    want[3] = want[0]
    for src, dst, rows in (([0, 5], [3, 1], None), ([0, 1], [3, 5], None), ([0, 1], [3, 2], [4, 5]), ([0, 1], [3, 2], [4, -1])):
        got, status = p.clone(), _status()
        K.kda_pool_copy(got, _i32(src).cuda(), _i32(dst).cuda(), rows=None if rows is None else _i32(rows).cuda(),
                        device_status=status)
        assert status.item() == 1
        assert torch.equal(got, want)
    # an entry that one pool has and another has not
    small, status = p[:4].clone(), _status()
    big = p.clone()
    K.kda_pool_copy([small, big], _i32([0]).cuda(), _i32([4]).cuda(), device_status=status)
    assert status.item() == 1 and torch.equal(small, p[:4]) and torch.equal(big[4], p[0])


def test_copy_nothing():
    p = torch.ones(5, 4, 8, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    K.kda_pool_copy(p, none, none)
    K.kda_pool_copy([], _i32([1]).cuda(), _i32([2]).cuda())
    assert bool((p == 1).all())


def test_copy_offsets_past_32_bits():
    p = torch.zeros(5000, 1 << 20, dtype=torch.uint8, device="cuda")
    p[4999] = 3
    K.kda_pool_copy(p, _i32([4999, 0]).cuda(), _i32([4500, 4998]).cuda())
    assert bool((p[4500] == 3).all()) and bool((p[4998] == 0).all()) and int(p[4501:4999].max()) == 0


# ---------------------------------------------------------------- the commit of accepted nodes
def _commit_case(seed, ctx, paths, nodes, shapes, dtype, views=None):
    g = _gen(seed)
    R, page = len(ctx), shapes[0][1]
    need = [(c + nodes + page - 1) // page for c in ctx]
    table = torch.zeros((R, max(need)), dtype=torch.int32)
    order, at = torch.randperm(sum(need) + 1, generator=g).to(torch.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    caches = [_rand(g, (sum(need) + 1, *s[1:]), dtype) for s in shapes]
    path = torch.full((R, nodes), -9, dtype=torch.int32)
    for r, p in enumerate(paths):
        path[r, :len(p)] = _i32(p)
    want = [c.clone() for c in caches]
    for r, p in enumerate(paths):
        for j, node in enumerate(p):
            a, b = ctx[r] + node, ctx[r] + j
            for w, c in zip(want, caches):
                w[int(table[r, b // page]), b % page] = c[int(table[r, a // page]), a % page]
    dev = [c.cuda() for c in caches]
    status = _status()
    seen = dev if views is None else [v(d) for v, d in zip(views, dev)]
    K.kda_cache_commit(seen, table.cuda(), _i32(ctx).cuda(), path.cuda(), _i32([len(p) for p in paths]).cuda(),
                       device_status=status)
    assert status.item() == 0
    for d, w in zip(dev, want):
        assert torch.equal(d.cpu(), w)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("heads,dim", [(2, 128), (8, 128), (1, 8), (3, 64)])
def test_commit_paths(dtype, page, heads, dim):
    paths = [[0, 1, 2], [], [1, 3, 4, 6], [7], [0, 2], [1, 2, 3, 4, 5, 6, 7]]
    _commit_case(30, [0, 5, 63, 64, 100, 15], paths, 8, [(0, page, heads, dim)] * 4, dtype)


def test_commit_long_paths_and_many_requests():
    _commit_case(31, [33], [list(range(1, 256))], 256, [(0, 16, 8, 128)] * 2, BF16)
    _commit_case(32, [3], [[i for i in range(250) if i % 3 != 1]], 256, [(0, 64, 16, 256), (0, 64, 1, 8)], BF16)
    paths = [[i for i in range(16) if (i * 7 + r) % 3] for r in range(300)]
    _commit_case(33, [(r * 13) % 70 for r in range(300)], paths, 16, [(0, 16, 2, 64)] * 3, BF16)


def test_commit_many_caches_and_layouts():
    paths = [[1, 2, 5], [0, 3]]
    _commit_case(34, [14, 2], paths, 6, [(0, 16, 2, 64)] * 100, BF16)
    _commit_case(35, [14, 2], paths, 6, [(0, 16, 4, 64), (0, 16, 96)], BF16)
    # heads before rows
    g = _gen(36)
    base = _rand(g, (4, 3, 16, 64), BF16).cuda()
    want = base.clone()
    want[2, :, 14] = base[2, :, 15]
    want[2, :, 15] = base[0, :, 1]
    K.kda_cache_commit(base.permute(0, 2, 1, 3), _i32([[2, 0]]).cuda(), _i32([14]).cuda(), _i32([[1, 3]]).cuda(), _i32([2]).cuda())
    assert torch.equal(base, want)


def test_commit_reports_what_only_the_device_sees():
    g = _gen(37)
    base = _rand(g, (6, 16, 2, 64), BF16).cuda()
    table, ctx = _i32([[0, 1, 2], [3, 4, 5]]), [10, 7]

    def run(path, accepted, ctx=ctx, table=table):
        got, status = base.clone(), _status()
        K.kda_cache_commit([got], table.cuda(), _i32(ctx).cuda(), _i32(path).cuda(), _i32(accepted).cuda(), device_status=status)
        return got, status.item()

    good = base.clone()
    good[3, 7] = base[3, 8]
    first = [1, 0, 0]
    for path, accepted, kw in (([[2, 2, 3], first], [2, 1], {}), ([[3, 2, 3], first], [2, 1], {}), ([[-1, 2, 3], first], [2, 1], {}),
                               ([[1, 2, 3], first], [4, 1], {}), ([[1, 2, 3], first], [-1, 1], {}),
                               ([[1, 2, 38], first], [3, 1], {}), ([[1, 2, 3], first], [2, 1], dict(ctx=[-1, 7])),
                               ([[1, 2, 2**31 - 1], first], [3, 1], {}),
                               ([[1, 2, 3], first], [2, 1], dict(ctx=[2**31 - 2, 7]))):
        got, st = run(path, accepted, **kw)
        assert st == 1 and torch.equal(got, good), (path, accepted, kw)
    # a page outside the pool: its rows alone stay
    got, st = run([[1, 6, 8], [0, 0, 0]], [3, 0], table=_i32([[0, 6, 2], [3, 4, 5]]))
    want = base.clone()
    want[0, 10] = base[0, 11]
    assert st == 1 and torch.equal(got, want)


def test_commit_after_a_verified_tree():
    """A tree's verification, the commit of its accepted path, and the next step over the
    longer context: as if the accepted tokens alone had been written."""
    R, N, Hq, Hk, D, page = 2, 6, 4, 2, 64, 16
    ctx = [37, 5]
    g = _gen(38)
    pages = 8
    table = torch.randperm(pages, generator=g).to(torch.int32).view(2, 4)
    kc, vc = _rand(g, (pages, page, Hk, D), BF16).cuda(), _rand(g, (pages, page, Hk, D), BF16).cuda()
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2], [-1, -1, 1, 1, 3, 0]])
    accepted = [[0, 1, 4], [1, 3, 4]]
    path = _i32([a + [0] * (N - len(a)) for a in accepted])
    ln = _i32(ctx).cuda()
    q = _rand(g, (R, N, Hq, D), BF16).cuda()
    tree = K.kda_tree_attention(q, kc, vc, table.cuda(), ln, tree_mask=K.tree_mask(parents.cuda()))
    K.kda_cache_commit([kc, vc], table.cuda(), ln, path.cuda(), _i32([3, 3]).cuda())
    # the accepted nodes as a chunk of new tokens behind the same context
    rows = torch.stack([q[r, a] for r, a in enumerate(accepted)])
    chunk = K.kda_chunk_attention(rows, kc, vc, table.cuda(), ln)
    out, ob, _, _ = chunk_reference(rows.flatten(0, 1).cpu(), kc.cpu(), vc.cpu(), table, ctx, [3, 3])
    within(chunk.flatten(0, 1), out, ob)
    within(torch.stack([tree[r, a] for r, a in enumerate(accepted)]).flatten(0, 1), out, ob)

"""Chunk attention, pool copies and the operators' status word on the GPU at the edges: the
walk over the line of work in several waves, scores that are all minus infinity, empty
pools, errors after a timeout."""
import math

import pytest
import torch

import kda_chunked_prefill_02_gb300 as K
from kda_chunked_prefill_02_gb300 import inputs
from ops_test_util import F64, U32, UNIT, rounding, within
from serve_edges_util import waves_of
from serve_test_util import chunk_reference

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
KDA_ERR_TIMEOUT = 4
# tokens a page table has room for: enough for the tensor-core kernel, whatever the lengths
ROOM = 300000


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _word(value=0):
    return torch.full((1,), value, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- the status word
def _reports():
    """Calls that report a length, an entry or a page, by name: functions of the status word."""
    g = _gen(1)
    calls = {}
    x, w = _rand(g, (4, 6, 128), BF16).cuda(), _rand(g, (128, 4), F32).cuda()
    state = _rand(g, (4, 3, 128), BF16).cuda()
    calls["conv slot"] = lambda s: K.kda_short_conv(x, w, conv_state=state.clone(), slot=_i32([0, 4, 2, 3]).cuda(), device_status=s)
    calls["conv lengths"] = lambda s: K.kda_short_conv(x.view(24, 128), w, cu_seqlens=_i32([0, 6, 4, 24]).cuda(), device_status=s)
    freq, _ = K.rope_frequencies(64, device="cuda")
    qr, kr = _rand(g, (5, 2, 64), BF16).cuda(), _rand(g, (5, 1, 64), BF16).cuda()
    cache = torch.zeros(2, 16, 1, 64, dtype=BF16, device="cuda")
    calls["rope slot"] = lambda s: K.kda_qk_norm_rope(qr, kr, torch.arange(5, dtype=torch.int32, device="cuda"), freq,
                                                      k_cache=cache.clone(), slots=torch.tensor([0, 1, 32, 3, 4]).cuda(),
                                                      device_status=s)
    kc, vc = _rand(g, (12, 16, 1, 64), BF16).cuda(), _rand(g, (12, 16, 1, 64), BF16).cuda()
    lens = _i32([30, 20]).cuda()
    for room in (64, ROOM):
        table = torch.zeros(2, room // 16, dtype=torch.int32)
        table[:, :4] = torch.arange(8, dtype=torch.int32).view(2, 4)
        page = table.clone()
        page[1, 0] = 12
        q = _rand(g, (2, 8, 24, 64), BF16).cuda()
        kind = "rows" if room == 64 else "tensor"
        assert K.chunk_attention_schedule(q, kc, table, packed=False)["kernel"] == kind
        for name, tab, ln in (("page", page.cuda(), lens), ("length", table.cuda(), _i32([30, -1]).cuda())):
            calls["chunk %s %s" % (kind, name)] = lambda s, t=tab, n=ln, q=q: K.kda_chunk_attention(q, kc, vc, t, n, device_status=s)
            calls["tree %s %s" % (kind, name)] = lambda s, t=tab, n=ln, q=q: K.kda_tree_attention(q, kc, vc, t, n, device_status=s)
    pool = torch.zeros(4, 16, 1, 64, dtype=BF16, device="cuda")
    calls["copy"] = lambda s: K.kda_pool_copy(pool, _i32([0]).cuda(), _i32([4]).cuda(), device_status=s)
    tab = _i32([[0, 1]]).cuda()
    for name, path, t in (("path", [[1, 1]], tab), ("page", [[1, 2]], _i32([[4, 1]]).cuda()), ("count", [[1, 2]], tab)):
        calls["commit " + name] = lambda s, p=path, t=t, n=3 if name == "count" else 2: K.kda_cache_commit(
            pool, t, _i32([3]).cuda(), _i32(p).cuda(), _i32([n]).cuda(), device_status=s)
    return calls


def test_a_timeout_is_kept():
    """A status word shared by a step's calls: what a later one reports (1) does not replace the
    timeout of one before (4), whose results are not all there."""
    for name, call in _reports().items():
        for before, after in ((0, 1), (KDA_ERR_TIMEOUT, KDA_ERR_TIMEOUT)):
            status = _word(before)
            call(status)
            assert status.item() == after, name


@pytest.mark.parametrize("op", ["chunk", "tree"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_timeout_and_bad_pages_in_one_call(op, D):
    """Waits that run out in some CTAs, pages outside the pool in others, in any order."""
    R, N = 60, 40
    kc = torch.randn(500, 16, 2, D, device="cuda").to(BF16)
    vc = torch.randn_like(kc)
    g = _gen(2)
    table = torch.randint(0, 520, (R, ROOM // 16), generator=g).to(torch.int32).cuda()   # one in 26 is none
    q, lens = _rand(g, (R, N, 8, D), BF16).cuda(), _i32([100 + 331 * (i % 13) for i in range(R)]).cuda()
    call = K.kda_chunk_attention if op == "chunk" else K.kda_tree_attention
    for limit in (2000, 20000, 200000):
        status = _word()
        with K.overrides(wait_limit_ns=limit, timeout_probe=True):
            call(q, kc, vc, table, lens, device_status=status)
        torch.cuda.synchronize()
        assert status.item() == KDA_ERR_TIMEOUT
    status = _word()
    call(q, kc, vc, table, lens, device_status=status)
    assert status.item() == 1


@pytest.mark.parametrize("kernel", ["sequential", "tensor"])
def test_a_timeout_is_kept_by_the_verification_of_drafts(kernel):
    """kda_verify with counts that no draft has: in a word that holds a timeout, and beside waits
    that run out in other CTAs."""
    d = inputs.verify_inputs(1206, R=400, D=6, H=4).to("cuda")
    accepted = d.accepted.clone()
    accepted[::2] = 7

    def run(status):
        K.kda_verify(d.q, d.k, d.v, d.g, d.beta, d.state_pool.clone(), accepted, device_status=status)
        torch.cuda.synchronize()
        return status.item()

    with K.overrides(verify_kernel=kernel):
        assert run(_word()) == 1 and run(_word(KDA_ERR_TIMEOUT)) == KDA_ERR_TIMEOUT
    if kernel == "tensor":
        for limit in (2000, 20000):
            with K.overrides(verify_kernel=kernel, wait_limit_ns=limit, timeout_probe=True):
                assert run(_word()) == KDA_ERR_TIMEOUT


# ---------------------------------------------------------------- pools
@pytest.mark.parametrize("shape", [(5, 4, 0, 64), (5, 4, 3, 0, 64)])
def test_copy_of_rows_that_hold_nothing(shape):
    """A pool of empty rows beside others has the rows it has: its first ones are nothing to copy,
    and nothing to report; a row count past them is, as for any pool."""
    empty = torch.empty(shape, dtype=F32, device="cuda")
    pool = torch.arange(5 * 4 * 8, dtype=torch.int32, device="cuda").view(5, 4, 8)
    want = pool.clone()
    want[3, :2] = want[0, :2]
    want[4] = want[1]
    src, dst, status = _i32([0, 1]).cuda(), _i32([3, 4]).cuda(), _word()
    K.kda_pool_copy([empty, pool], src, dst, rows=_i32([2, 4]).cuda(), device_status=status)
    assert status.item() == 0 and torch.equal(pool, want)
    K.kda_pool_copy([empty, pool], src, dst, device_status=status)
    assert status.item() == 0
    K.kda_pool_copy(empty, src, dst, rows=_i32([5, 4]).cuda(), device_status=status)
    assert status.item() == 1


# ---------------------------------------------------------------- scores that are minus infinity
def _one_request(seed, ctx, new, Hq, Hk, D, page, dtype, room):
    """q, caches, a page table and lengths of one request, on the host."""
    g = _gen(seed)
    pages = (ctx + new + page - 1) // page
    table = torch.zeros(1, max(pages, room // page), dtype=torch.int32)
    table[0, :pages] = torch.randperm(pages, generator=g).to(torch.int32)
    return (_rand(g, (new, Hq, D), dtype, 1.5), _rand(g, (pages, page, Hk, D), dtype), _rand(g, (pages, page, Hk, D), dtype),
            table, _i32([ctx]))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx,new,hidden", [(0, 200, 48), (0, 3, 16), (100, 1, 96), (100, 30, 144), (6000, 1, 6000), (6000, 300, 5008),
                                            (40000, 1, 40000), (40000, 20, 48000)])
def test_chunk_scores_that_are_minus_infinity(dtype, room, D, ctx, new, hidden):
    """The first `hidden` keys have a component of minus infinity that every query meets with 1: a
    token that sees others beside them sees those alone, one that sees no others is 0 / 0."""
    page, n = 16, min(hidden, ctx + new)
    q, kc, vc, table, lens = _one_request(4, ctx, new, 4, 1, D, page, dtype, room)
    q[..., 5] = 1
    kind = K.chunk_attention_schedule(q, kc, table)["kernel"]
    assert kind == "tensor" or room == 0
    kc[table[0, :(n + page - 1) // page].long(), :, :, 5] = -math.inf
    got, lse = K.kda_chunk_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(),
                                     cu_seqlens=_i32([0, new]).cuda(), return_lse=True)
    got, lse = got.cpu(), lse.cpu()
    gone = max(0, min(new, hidden - ctx))      # tokens that see nothing else
    assert bool(torch.isnan(got[:gone]).all()) and bool((lse[:gone] == -math.inf).all())
    if gone < new:   # the others as over a context without those keys
        out, ob, want, lb = chunk_reference(q[gone:], kc, vc, table[:, hidden // page:], [ctx + gone - hidden], [new - gone])
        within(got[gone:], out, ob)
        within(lse[gone:], want, lb)


# ---------------------------------------------------------------- the line of work in waves
def _reference(q, kc, vc, table, ctx, new, start):
    """chunk_reference (serve_test_util.py) of one request on the GPU, a key head and 256 rows at a
    time, for values that are all finite: out, its bound [new, Hq, D], log-sums, theirs."""
    Hq, D = q.shape[1:]
    page, Hk = kc.shape[1], kc.shape[2]
    G, L, unit = Hq // Hk, ctx + new, UNIT[q.dtype]
    at = torch.arange(L, device="cuda")
    pages = table.long()[at // page]
    out, bound = (torch.empty(new, Hq, D, dtype=F64, device="cuda") for _ in range(2))
    lse, lse_bound = (torch.empty(new, Hq, dtype=F64, device="cuda") for _ in range(2))
    summed = (L + 16) * U32
    for h in range(Hk):
        k, v = (c[pages, at % page, h].to(F64) for c in (kc, vc))
        for i in range(0, new, 256 // min(G, 256)):
            x = q[start + i:start + min(i + 256 // min(G, 256), new), h * G:(h + 1) * G].to(F64)   # [n, G, D]
            n = x.shape[0]
            sees = (at[None] <= ctx + i + torch.arange(n, device="cuda")[:, None])[:, None]        # [n, 1, L]
            s = torch.where(sees, x @ k.t() * D ** -0.5, -math.inf)
            p = torch.softmax(s, -1)
            y, near = p @ v, p @ v.abs()
            mag = torch.where(sees, x.abs() @ k.abs().t(), 0).amax(-1)
            top = torch.where(sees, s, 0).abs().amax(-1)
            ds = (D + 8) * U32 * D ** -0.5 * mag + top * 2.0 ** -21 + 2.0 ** -20
            b = near * (unit + 2 * ds + 2 * summed)[..., None] * (1 + unit) + rounding(y, q.dtype) * (1 + unit)
            z, heads = torch.logsumexp(s, -1), slice(h * G, (h + 1) * G)
            out[i:i + n, heads], bound[i:i + n, heads], lse[i:i + n, heads] = y, b, z
            lse_bound[i:i + n, heads] = ds + summed + z.abs() * 2.0 ** -21 + 2.0 ** -20
    return out.cpu(), bound.cpu(), lse.cpu(), lse_bound.cpu()


@pytest.mark.parametrize("dtype,Hq,Hk,D,page,ctx,new,waves,form", [
    (BF16, 32, 8, 128, 64, [30000], [1024], 2, "packed"),
    (BF16, 32, 8, 128, 16, [126976], [700], 8, "packed"),
    (F16, 16, 16, 64, 16, [60000], [1500], 4, "packed"),
    (BF16, 16, 4, 256, 64, [50000], [900], 4, "packed"),
    (F16, 32, 4, 128, 128, [70011], [333], 2, "in place"),
    (BF16, 32, 8, 128, 64, [0, 20000, 3, 9000, 100, 40, 2500, 0], [900, 700, 0, 600, 1, 1, 33, 1], 2, "packed"),
    (BF16, 32, 8, 128, 64, [25000, 24000], [800, 800], 4, "padded")])
def test_chunk_in_waves(dtype, Hq, Hk, D, page, ctx, new, waves, form):
    """Every row of calls whose line of work is walked in several waves against 64 bits: items cut
    between two CTAs and between two waves, the requests walked again in each.  A part of an
    item's keys that is lost or counted twice shows in the log-sums, a part of its values in
    channels whose mean is 1 or -1 by a bit of the position."""
    g = torch.Generator("cuda").manual_seed(3)

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sms != 152 or waves_of(ctx, new, Hk, Hq // Hk, D, sms) == waves
    need = [(c + n + page - 1) // page for c, n in zip(ctx, new)]
    kc, vc = rand(sum(need), page, Hk, D), rand(sum(need), page, Hk, D)
    table = torch.zeros(len(ctx), max(need), dtype=torch.int32, device="cuda")
    order, at = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
        pos = torch.arange(n * page, device="cuda")
        mean = 2 * ((pos[:, None] >> (torch.arange(D, device="cuda") % 9 + 7)) & 1) - 1
        vc[table[r, :n].long()] += mean.view(n, page, 1, D).to(dtype)
    q, lens, cu = rand(sum(new), Hq, D, scale=1.5), _i32(ctx).cuda(), _i32([0] + new).cumsum(0).to(torch.int32)
    shaped = q.view(len(ctx), -1, Hq, D) if form == "padded" else q
    cut = K.chunk_attention_schedule(shaped, kc, table, packed=form != "padded")
    assert cut["kernel"] == "tensor"
    # the workspace begins with what each stretch of a wave left in its two slots: a state (0: nothing) and an item
    ws = torch.zeros(cut["ctas"] * 2 * (16 + 256 * (D + 1) * 4), dtype=torch.uint8, device="cuda")
    status = _word()
    x = shaped.clone()
    got, lse = K.kda_chunk_attention(x, kc, vc, table, lens, cu_seqlens=None if form == "padded" else cu.cuda(), workspace=ws,
                                     out=x if form == "in place" else None, return_lse=True, device_status=status)
    assert status.item() == 0
    states = ws[:cut["ctas"] * 32].view(torch.int32).view(-1, 2, 4)[:, :, 0]
    used = int(states.any(1).nonzero().max()) // (sms // 2 if D == 256 else sms) + 1
    assert used == waves_of(ctx, new, Hk, Hq // Hk, D, sms)
    got, lse = got.view(-1, Hq, D), lse.view(-1, Hq)
    for r, (c, n) in enumerate(zip(ctx, new)):
        if n > 0:
            a = int(cu[r])
            want, bound, lse_want, lse_bound = _reference(q, kc, vc, table[r], c, n, a)
            within(got[a:a + n], want, bound)
            within(lse[a:a + n], lse_want, lse_bound)

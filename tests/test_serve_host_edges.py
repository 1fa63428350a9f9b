"""Host side of chunk attention at the edges (no GPU): the room for waves over its line of work."""
import ctypes
import random

import pytest
import torch

from serve_edges_util import waves_of

PTR = 1 << 20   # never dereferenced


@pytest.fixture(scope="module")
def ops():
    from kda_chunked_prefill_02_gb300 import build, ops as o
    build.build()
    o._fn()
    return o


def _args(ops, R, T, Hq, Hk, D, tokens, max_context=-1, packed=True):
    a = ops.ChunkAttentionArgs()
    a.q = a.k_cache = a.v_cache = a.page_table = a.context_lens = PTR
    a.out, a.cu_seqlens = 2 * PTR, PTR if packed else None
    for n in ("q", "out", "k_cache", "v_cache"):
        for i, s in enumerate((T * Hq * D, Hq * D, D)):
            setattr(a, "%s_stride%d" % (n, i), s)
    a.num_requests, a.seqlen, a.num_q_heads, a.num_k_heads, a.head_dim = R, T, Hq, Hk, D
    a.num_pages, a.page_size, a.pages_per_request, a.scale, a.max_context = 100, 16, tokens // 16, 0.1, max_context
    return a


def _stretches(ops, a, num_sms):
    s = ops.ChunkSchedule()
    assert ops._fn().kda_chunk_attention_schedule(ctypes.byref(a), num_sms, ctypes.byref(s)) == 0
    return s.ctas if s.kernel == 1 else 0


def test_chunk_room_for_waves(ops):
    """Room for the waves that a call may walk, not for eight wherever a context is long."""
    def waves(*shape, **kw):
        n = _stretches(ops, _args(ops, *shape, **kw), 152)
        assert n % (76 if shape[4] == 256 else 152) == 0
        return n // (76 if shape[4] == 256 else 152)
    assert waves(1, 2048, 32, 8, 128, 129024) == 8                    # a piece far from its prompt's begin
    assert waves(1, 2048, 32, 8, 128, 1 << 20, max_context=126976) == 8
    assert waves(64, 2108, 32, 8, 128, 4608) == 1                     # single tokens and a few pieces
    assert waves(24, 12011, 16, 16, 64, 1024) == 1                    # ragged prompts
    assert waves(64, 64, 32, 8, 128, 1 << 20) == 1                    # single tokens, however long
    assert waves(1, 8192, 32, 8, 128, 8192) == 1                      # K and V stay in L2
    assert waves(1, 32768, 32, 8, 128, 32768) == 2
    assert waves(2, 800, 32, 8, 128, 26000, packed=False) == 4
    assert waves(1, 900, 16, 4, 256, 50900) == 4


def test_chunk_workspace_with_waves(ops):
    """Two items a stretch of every wave, 256 rows of values and log-sums each."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152
    for D, Hq, Hk in ((64, 16, 16), (128, 32, 8), (256, 16, 4)):
        for R, T, tokens in ((1, 2048, 129024), (64, 2108, 4608), (1, 8192, 8192)):
            a = _args(ops, R, T, Hq, Hk, D, tokens)
            n = _stretches(ops, a, sms)
            assert n > 0 and ops._fn().kda_chunk_attention_workspace_size(ctypes.byref(a)) == 2 * n * (16 + 256 * (D + 1) * 4)


def test_chunk_room_holds_the_waves_of_any_lengths(ops):
    """Whatever the lengths on the device are, the waves that the kernel walks have room, so that
    the room never decides."""
    rng, reached = random.Random(5), set()
    for _ in range(3000):
        D, Hk, G = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 7, 8, 16, 64])
        R, packed = int(2 ** rng.uniform(0, 6)), rng.random() < 0.7
        top = int(2 ** rng.uniform(8, 18))
        new = [min(top, rng.choice([1, 1, 40, 300, 1000, 5000]) * rng.randint(1, 3)) for _ in range(R)]
        if rng.random() < 0.2:
            new = [0 if rng.random() < 0.5 else n for n in new]
        if not packed:
            new = [max(1, new[0])] * R
        ctx = [rng.choice([0, top - n, rng.randint(0, top - n)]) for n in new]
        T, sms = sum(new) if packed else new[0], rng.choice([152, 152, 148, 20])
        if T == 0:
            continue
        a = _args(ops, R, T, Hk * G, Hk, D, max(16, (top + 15) // 16 * 16),
                  max_context=max(ctx) if rng.random() < 0.5 else -1, packed=packed)
        room, one = _stretches(ops, a, sms), sms // 2 if D == 256 else sms
        if room:
            need = waves_of(ctx, new, Hk, G, D, sms)
            assert need <= room // one <= 8, (ctx, new, Hk, G, D, sms)
            reached.add(need)
    assert reached == set(range(1, 9))

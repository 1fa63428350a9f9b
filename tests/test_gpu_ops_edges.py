"""The operators of include/kda_ops.h on the GPU at the edges of what their headers allow."""
import pytest
import torch

import kda_chunked_prefill_02_gb300 as K
from ops_test_util import rope_reference, within

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


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

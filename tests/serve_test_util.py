"""Plain 64-bit forms of chunk attention and the residual stream's norm, with the error
each kernel may make, derived from the number formats and the instructions used."""
import math

import torch

from ops_test_util import F64, U32, UNIT, rounding


def chunk_reference(q, k_cache, v_cache, table, ctx, new, *, scale=None):
    """q [T, Hq, D], requests of new[r] rows one after the other.  Returns (out, out
    bound, lse, lse bound); what a row does not see has no part in it, whatever it holds."""
    T, Hq, D = q.shape
    page, Hk = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    unit = UNIT[q.dtype]
    out, ob = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    lse, lb = torch.full((T, Hq), -math.inf, dtype=F64), torch.zeros((T, Hq), dtype=F64)
    start = 0
    for r, n in enumerate(new):
        if n == 0:
            continue
        c = int(ctx[r])
        at = torch.arange(c + n)
        pages = table[r].long()[at // page]
        k = k_cache[pages, at % page].to(F64).permute(1, 0, 2)     # [Hk, L, D]
        v = v_cache[pages, at % page].to(F64).permute(1, 0, 2)
        sees = at[None, :] <= c + torch.arange(n)[:, None]         # [n, L]
        x = q[start:start + n].to(F64).reshape(n, Hk, G, D).permute(1, 2, 0, 3)   # [Hk, G, n, D]
        s = (x @ k[:, None].transpose(-1, -2)) * scale
        s = torch.where(sees, s, torch.full_like(s, -math.inf))
        p = torch.softmax(s, -1)
        # (0 times a value that is not finite would be one)
        bad = ~torch.isfinite(v)
        vf = torch.where(bad, torch.zeros_like(v), v)
        y, near = p @ vf[:, None], p @ vf.abs()[:, None]
        if bool(bad.any()):
            hit = torch.where(bad, v, torch.zeros_like(v))
            for h in range(Hk):
                for j in torch.nonzero(bad[h].any(-1)).flatten().tolist():
                    y[h, :, max(0, j - c):] += hit[h, j]
        # a score: D products and sums in fp32, scaled; the exponential: 2^-21 and the
        # rounding of its argument; the sums over the keys
        ks = torch.where(torch.isfinite(k), k, torch.zeros_like(k)).abs()
        mag = torch.where(sees, x.abs() @ ks[:, None].transpose(-1, -2), torch.zeros_like(s)).amax(-1)
        top = torch.where(sees, s, torch.zeros_like(s)).abs().amax(-1)
        ds = (D + 8) * U32 * abs(scale) * mag + top * 2.0 ** -21 + 2.0 ** -20
        summed = (c + n + 16) * U32
        b = near * (unit + 2 * ds + 2 * summed)[..., None] * (1 + unit) + rounding(y, q.dtype) * (1 + unit)
        out[start:start + n] = y.permute(2, 0, 1, 3).reshape(n, Hq, D)
        ob[start:start + n] = b.permute(2, 0, 1, 3).reshape(n, Hq, D)
        z = torch.logsumexp(s, -1)
        lse[start:start + n] = z.permute(2, 0, 1).reshape(n, Hq)
        lb[start:start + n] = (ds + summed + z.abs() * 2.0 ** -21 + 2.0 ** -20).permute(2, 0, 1).reshape(n, Hq)
        start += n
    return out, ob, lse, lb


def residual_reference(x, y, *, weight=None, post_norm=False, post_weight=None, gate=None, gate_sigmoid=False,
                       alpha=1.0, norm_eps=1e-6, dtype=None):
    """Returns (h, bound, new x, bound) in fp64."""
    E = x.shape[-1]
    dtype = dtype or (y.dtype if y is not None else x.dtype)
    eps = float(torch.tensor(norm_eps, dtype=torch.float32))
    one = torch.ones(E, dtype=F64)
    # a mean square: sums of positive terms over 16 elements, two pieces and 10 exchanges, some
    # 32 roundings at most, halved by the root; its division, eps, the root (2^-22), 2 products
    rel = 2.0 ** -19
    v = x.to(F64)
    ex = torch.zeros_like(v)
    if y is not None:
        u = y.to(F64)
        eu = torch.zeros_like(u)
        if post_norm:
            u = u * (u.square().mean(-1, keepdim=True) + eps).rsqrt() * (one if post_weight is None else post_weight.to(F64))
            eu = u.abs() * rel
        if gate is not None:
            g = gate.to(F64)
            if gate_sigmoid:
                # the exponential (2^-22) of a rounded product, the sum, the reciprocal (2^-23)
                eg = 2.0 ** -20 + g.abs() * 2.0 ** -22
                g = torch.sigmoid(g)
            else:
                eg = 0.0
            eu = eu * g.abs() + (u * g).abs() * (eg + U32)
            u = u * g
        a = float(torch.tensor(alpha, dtype=torch.float32))
        v = v + a * u
        ex = abs(a) * eu + v.abs() * U32
    norm = (v.square().mean(-1, keepdim=True) + eps).sqrt()
    w = one if weight is None else weight.to(F64)
    h = v / norm * w
    # the row's own error moves its norm by the error's at most
    eh = ex / norm * w.abs() + h.abs() * (rel + ex.square().mean(-1, keepdim=True).sqrt() / norm)
    xr = U32 * v.abs() if x.dtype == torch.float32 else rounding(v, x.dtype)
    return h, eh + rounding(h, dtype) * (1 + 2.0 ** -8), v, ex + xr * (1 + 2.0 ** -8)

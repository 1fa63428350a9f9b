"""Plain 64-bit forms of the operators in include/kda_ops.h, with the error each
kernel may make, derived from the number formats and the instructions used."""
import math

import torch

F64 = torch.float64
# Unit roundoff of the element types (half a unit in the last of 8 / 11 bits) and
# half the spacing of fp16's subnormals.
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
U32 = 2.0 ** -24


def rounding(y, dtype):
    """One rounding of y to dtype."""
    return UNIT[dtype] * y.abs() + TINY[dtype]


def conv_reference(x, weight, *, bias=None, state=None, starts, lengths, slots=None, has_state=None, accepted=None,
                   silu=True, norm_channels=0, norm_eps=1e-6):
    """x [tokens, C] (flat), sequences at starts/lengths.  Returns (y, bound, new state)
    in fp64; `bound` is the error a fp32 evaluation rounded once may have."""
    C, W = weight.shape
    w, xs = weight.to(F64), x.to(F64)
    y = torch.zeros(x.shape, dtype=F64)
    bound = torch.zeros(x.shape, dtype=F64)
    new = None if state is None else state.clone()
    for n, (s, length) in enumerate(zip(starts, lengths)):
        old = torch.zeros((W - 1, C), dtype=x.dtype)
        slot = n if slots is None else int(slots[n])
        if state is not None and (has_state is None or int(has_state[n])):
            old = state[slot]
        ext = torch.cat([old, x[s:s + length]])
        if new is not None:
            a = length if accepted is None else int(accepted[n])
            new[slot] = ext[a:a + W - 1]
        ext = ext.to(F64)
        z = torch.zeros((length, C), dtype=F64) if bias is None else bias.to(F64).expand(length, C).clone()
        mag = z.abs()
        for j in range(W):
            z = z + ext[j:j + length] * w[:, j]
            mag = mag + (ext[j:j + length] * w[:, j]).abs()
        # W fused multiply-adds: (W + 1) roundings of sums no larger than mag
        err = (W + 1) * U32 * mag
        if silu:
            v = z * torch.sigmoid(z)
            # |silu'| <= 1.1; e^-z: 2^-22 and the rounding of its argument (|z| log2 e),
            # the sum, the product, the reciprocal (2^-23) and three products
            err = 1.1 * err + v.abs() * (2.0 ** -19 + z.abs() * 2.0 ** -22) + 2e-17 * z.abs()
        else:
            v = z
        if norm_channels:
            h = v[:, :norm_channels].reshape(length, norm_channels // 128, 128)
            e = err[:, :norm_channels].reshape(length, norm_channels // 128, 128)
            norm = (h.square().sum(-1, keepdim=True) + norm_eps).sqrt()
            # the head's own error moves the norm by |e| at most; 128 squares, the root (2^-22), the product
            he = e / norm + (h / norm).abs() * (e.norm(dim=-1, keepdim=True) / norm + 2.0 ** -18)
            v = torch.cat([(h / norm).reshape(length, norm_channels), v[:, norm_channels:]], 1)
            err = torch.cat([he.reshape(length, norm_channels), err[:, norm_channels:]], 1)
        y[s:s + length] = v
        bound[s:s + length] = err + rounding(v, x.dtype) * (1 + 2.0 ** -8)
    return y, bound, new


def rope_reference(x, positions, inv_freq, weight, *, norm=True, norm_eps=1e-6, interleaved=False, scale=1.0):
    """x [T, H, D]; returns (y, bound) in fp64."""
    v = x.to(F64)
    w = torch.ones(x.shape[-1], dtype=F64) if weight is None else weight.to(F64)
    if norm:
        v = v * (v.square().mean(-1, keepdim=True) + norm_eps).rsqrt()
    v = v * w
    # squares and their sum (256 channels over shuffles: 16 roundings), the division, the
    # root (2^-22), three products; trigonometry: the angle (1e-6) and sin / cos (2^-20)
    rel, trig = 2.0 ** -19, 1e-6 + 2.0 ** -20 + 2.0 ** -23
    y = v.clone()
    mag = torch.zeros_like(v)
    if inv_freq is not None:
        half = inv_freq.numel()
        angle = positions.to(F64)[:, None] * inv_freq.to(F64)
        c, s = (torch.cos(angle) * scale)[:, None], (torch.sin(angle) * scale)[:, None]
        ia = torch.arange(half) * 2 if interleaved else torch.arange(half)
        ib = ia + 1 if interleaved else ia + half
        a, b = v[..., ia], v[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * abs(scale)
    return y, mag * (trig + rel) + y.abs() * rel + rounding(y, x.dtype) * (1 + 2.0 ** -8)


def tree_reference(q, k_cache, v_cache, table, ctx, *, sees=None, nodes=None, scale=None):
    """q [R, N, Hq, D]; sees [R, N, N] bool (None: chain).  Returns (out, out bound, lse, lse bound)."""
    R, N, Hq, D = q.shape
    page, Hk = k_cache.shape[1], k_cache.shape[2]
    scale = D ** -0.5 if scale is None else scale
    unit = UNIT[q.dtype]
    out, ob = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    lse, lb = torch.full((R, N, Hq), -math.inf, dtype=F64), torch.zeros((R, N, Hq), dtype=F64)
    for r in range(R):
        c, n = int(ctx[r]), N if nodes is None else int(nodes[r])
        for i in range(n):
            see = torch.ones(c + n, dtype=torch.bool)
            see[c:] = (torch.arange(n) <= i) if sees is None else sees[r, i, :n]
            pos = torch.nonzero(see).flatten()
            if pos.numel() == 0:
                continue
            pages = table[r].long()[pos // page]
            k = k_cache[pages, pos % page].to(F64).repeat_interleave(Hq // Hk, 1)   # [L, Hq, D]
            v = v_cache[pages, pos % page].to(F64).repeat_interleave(Hq // Hk, 1)
            x = q[r, i].to(F64)
            s = torch.einsum("hd,lhd->hl", x, k) * scale
            p = torch.softmax(s, -1)
            y = torch.einsum("hl,lhd->hd", p, v)
            near = torch.einsum("hl,lhd->hd", p, v.abs())
            # a score: D products and sums in fp32, scaled; the exponential: 2^-21 and the
            # rounding of its argument; the sums over L keys
            ds = (D + 8) * U32 * abs(scale) * torch.einsum("hd,lhd->hl", x.abs(), k.abs()).amax(-1)
            ds = ds + s.abs().amax(-1) * 2.0 ** -21 + 2.0 ** -20
            summed = (pos.numel() + 16) * U32
            out[r, i] = y
            # a weight is rounded to the element type before it meets v
            ob[r, i] = near * (unit + 2 * ds + 2 * summed)[:, None] * (1 + unit) + rounding(y, q.dtype) * (1 + unit)
            lse[r, i] = torch.logsumexp(s, -1)
            lb[r, i] = ds + summed + lse[r, i].abs() * 2.0 ** -21 + 2.0 ** -20
    return out, ob, lse, lb


def within(got, want, bound):
    """Every element of got within bound of want (equal where the bound is 0); returns the worst ratio."""
    d = (got.to(F64).cpu() - want).abs()
    assert torch.isfinite(d).all()
    assert bool((d <= bound).all()), float((d / bound.clamp_min(1e-300)).max())
    return float((d / bound.clamp_min(1e-300)).max())

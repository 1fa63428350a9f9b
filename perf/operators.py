"""The operators around Kimi Delta Attention in a serving stack: cases, inputs, plain forms.

Three operators of a decoder that mixes KDA layers with softmax-attention layers:

* conv: the short causal convolution in front of a KDA layer (depthwise, SiLU,
  per-head L2 norm of its q and k channels), over prompts, drafts and single
  tokens, with the last inputs of every request kept in a pool;
* rope: RMS norm of every query and key head and the position rotation in one
  pass, the keys and values optionally put into their rows of a paged cache;
* tree: attention of a tree (or chain) of drafted tokens, or of a single token,
  over a paged cache.

With `own` false, run() computes them with elementary torch operations in 32
bits; with `own` true it calls this repository's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One request's next token in a two-head layer: the latency of the smallest call.
        {"name": "conv_token_r1", "op": "conv", "form": "token", "requests": 1, "tokens": 1, "heads": 2,
         "width": 4, "bias": False, "norm": True, "dtype": "bf16"},
        # A serving step: the next token of 256 requests in a 32-head layer.
        {"name": "conv_token_r256", "op": "conv", "form": "token", "requests": 256, "tokens": 1, "heads": 32,
         "width": 4, "bias": False, "norm": True, "dtype": "bf16"},
        # A packed batch of prompts of 8 lengths, some the continuation of an earlier piece.
        {"name": "conv_prompts_t32768", "op": "conv", "form": "packed", "requests": 8, "tokens": 32768, "heads": 32,
         "width": 4, "bias": False, "norm": True, "dtype": "bf16"},
        # Equal prompts of an odd length, fp16, three taps and a bias, no norm.
        {"name": "conv_padded_t2047", "op": "conv", "form": "padded", "requests": 5, "tokens": 2047, "heads": 10,
         "width": 3, "bias": True, "norm": False, "dtype": "fp16"},
        # One token of one request with few heads: latency.
        {"name": "rope_token_r1", "op": "rope", "tokens": 1, "q_heads": 8, "k_heads": 2, "dim": 128, "rot": 128,
         "interleaved": False, "scaled": False, "cache": 64, "dtype": "bf16"},
        # 256 requests x 4 drafts, keys and values into the cache, positions of long contexts.
        {"name": "rope_drafts_t1024", "op": "rope", "tokens": 1024, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "scaled": True, "cache": 64, "dtype": "bf16"},
        # A batch of prompts, interleaved rotation of half of the head, results in place of a cache.
        {"name": "rope_prompts_t32768", "op": "rope", "tokens": 32768, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 64,
         "interleaved": True, "scaled": False, "cache": 0, "dtype": "fp16"},
        # Wide heads with a quarter rotated, an odd number of tokens, into pages of 16.
        {"name": "rope_wide_t8191", "op": "rope", "tokens": 8191, "q_heads": 16, "k_heads": 2, "dim": 256, "rot": 64,
         "interleaved": False, "scaled": True, "cache": 16, "dtype": "bf16"},
        # One request's next token over a short context: latency.
        {"name": "tree_token_r1", "op": "tree", "requests": 1, "nodes": 1, "context": 1000, "q_heads": 8, "k_heads": 2,
         "dim": 128, "page": 64, "chain": True, "dtype": "bf16"},
        # The draft verification of 256 requests x 4 drafts over ragged contexts.
        {"name": "tree_chain_r256", "op": "tree", "requests": 256, "nodes": 4, "context": 4096, "q_heads": 32,
         "k_heads": 8, "dim": 128, "page": 64, "chain": True, "dtype": "bf16"},
        # Trees of 61 drafted tokens over ragged contexts in pages of 16.
        {"name": "tree_wide_r24", "op": "tree", "requests": 24, "nodes": 61, "context": 9000, "q_heads": 32,
         "k_heads": 4, "dim": 128, "page": 16, "chain": False, "dtype": "fp16"},
        # One request with a tree of 16 over a long context.
        {"name": "tree_long_r1", "op": "tree", "requests": 1, "nodes": 16, "context": 131072, "q_heads": 32,
         "k_heads": 8, "dim": 128, "page": 64, "chain": False, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["conv", "rope", "tree"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "conv":
        form = rng.choice(["token", "padded", "packed"])
        heads = rng.choice([1, 2, 4, 6, 10, 16, 20, 32])
        requests = _log_int(rng, 1, 512 if form == "token" else 32)
        most = max(requests, 32768 * 32 // heads // (1 if form == "packed" else requests))
        tokens = 1 if form == "token" else _log_int(rng, requests if form == "packed" else 2,
                                                    min(32768 if form == "packed" else 4096, most))
        return {"op": op, "form": form, "requests": requests, "tokens": tokens, "heads": heads,
                "width": rng.choice([2, 3, 4, 4]), "bias": rng.random() < 0.3, "norm": rng.random() < 0.7,
                "dtype": dtype}
    if op == "rope":
        dim, q_heads, k_heads = rng.choice([(64, 16, 16), (64, 20, 4), (96, 12, 3), (128, 8, 1), (128, 32, 8),
                                            (128, 40, 8), (256, 16, 2), (256, 8, 4)])
        rot = rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= dim])
        return {"op": op, "tokens": _log_int(rng, 1, 32768 * 40 * 128 // ((q_heads + 2 * k_heads) * dim) // 2),
                "q_heads": q_heads, "k_heads": k_heads, "dim": dim, "rot": rot, "interleaved": rng.random() < 0.4,
                "scaled": rng.random() < 0.5, "cache": rng.choice([0, 16, 64, 100]), "dtype": dtype}
    nodes = rng.choice([1, 1, 2, 4, 5, 8, 16, 31, 64])
    q_heads, k_heads, dim = rng.choice([(8, 2, 128), (32, 8, 128), (16, 16, 64), (32, 4, 128), (40, 8, 128),
                                        (16, 2, 256), (6, 6, 64)])
    requests = _log_int(rng, 1, 256)
    # no more keys and scores in all than the largest listed cases read and form
    most = int(0.7 * min(256 * 4096 * 8 * 128 // (k_heads * dim), 24 * 61 * 9000 * 32 * 128 // (nodes * q_heads * dim))) // requests
    return {"op": op, "requests": requests, "nodes": nodes, "context": _log_int(rng, 1, max(1, min(131072, most))),
            "q_heads": q_heads, "k_heads": k_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128, 24]),
            "chain": rng.random() < 0.4, "dtype": dtype}


def _lengths(requests, most):
    """Ragged context lengths, the first the longest: a fixed function of the case."""
    return [max(1, int(most * (1.0 if r == 0 else 0.2 + 0.8 * ((r * 0.6180339887) % 1.0)))) for r in range(requests)]


def _pieces(requests, tokens):
    """`tokens` cut into `requests` lengths of at least 1, uneven, one of them a single token."""
    if requests == 1:
        return [tokens]
    weight = [0.15 + (r * 0.6180339887) % 1.0 for r in range(requests - 1)]
    spare = tokens - requests
    take = [1 + int(spare * w / sum(weight)) for w in weight]
    take[0] += tokens - 1 - sum(take)
    return take + [1]


def _normal(gen, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if scale != 1.0 else dtype)
    return x if scale == 1.0 else (x * scale).to(dtype)


def _frequencies(rot, scaled):
    """Rotation frequencies (base 1e6); scaled: position interpolation by 8 of the slow half."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 1e6 ** (-2.0 * i / rot)
    if scaled:
        f = torch.where(i >= rot // 4, f / 8.0, f)
    return f.to(torch.float32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    host = torch.Generator().manual_seed(1000003 * seed + 29)
    dt = _DT[case["dtype"]]
    s = {"op": case["op"]}
    if case["op"] == "conv":
        n, t, w = case["requests"], case["tokens"], case["width"]
        c = 3 * case["heads"] * 128
        packed = case["form"] == "packed"
        s["x"] = _normal(gen, (t, c) if packed else (n, t, c), dt)
        s["weight"] = _normal(gen, (c, w), torch.float32, 1.0 / math.sqrt(w))
        s["bias"] = _normal(gen, (c,), torch.float32, 0.1) if case["bias"] else None
        s["pool"] = _normal(gen, (n + n // 2 + 1, w - 1, c), dt)
        s["slot"] = torch.randperm(n + n // 2 + 1, generator=host)[:n].to(torch.int32).cuda()
        s["has_state"] = None if case["form"] == "token" else (torch.arange(n) % 3 != 1).to(torch.int32).cuda()
        ends = [0]
        ends.extend(_pieces(n, t) if packed else [t] * n)
        s["cu"] = torch.tensor(ends).cumsum(0).to(torch.int32).cuda()
        s["packed"] = packed
        s["norm_channels"] = 2 * case["heads"] * 128 if case["norm"] else 0
        s["eps"] = 1e-6
    elif case["op"] == "rope":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        # q, k and v as a fused projection leaves them: three views of one row
        qkv = _normal(gen, (t, hq + 2 * hk, d), dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["positions"] = torch.randint(0, 131072, (t,), generator=host).to(torch.int32).cuda()
        s["freq"] = _frequencies(case["rot"], case["scaled"])
        s["scale"] = 0.1 * math.log(8.0) + 1.0 if case["scaled"] else 1.0
        s["q_weight"] = 1.0 + _normal(gen, (d,), torch.float32, 0.1)
        s["k_weight"] = 1.0 + _normal(gen, (d,), torch.float32, 0.1)
        s["interleaved"] = case["interleaved"]
        s["eps"] = 1e-6
        s["k_cache"] = s["v_cache"] = s["slots"] = None
        if case["cache"]:
            pages = (t + case["cache"] - 1) // case["cache"] + 1
            s["k_cache"] = torch.zeros((pages, case["cache"], hk, d), dtype=dt, device="cuda")
            s["v_cache"] = torch.zeros_like(s["k_cache"])
            s["slots"] = torch.randperm(pages * case["cache"], generator=host)[:t].cuda()
    else:
        r, n, hq, hk, d, page = (case[x] for x in ("requests", "nodes", "q_heads", "k_heads", "dim", "page"))
        lens = _lengths(r, case["context"])
        need = [(x + n + page - 1) // page for x in lens]
        order = torch.randperm(sum(need), generator=host).to(torch.int32)
        table = torch.zeros((r, max(need)), dtype=torch.int32)
        used = torch.arange(max(need))[None, :] < torch.tensor(need)[:, None]
        table[used] = order
        s["q"] = _normal(gen, (r, n, hq, d), dt, 1.5)
        s["k_cache"] = _normal(gen, (sum(need), page, hk, d), dt)
        s["v_cache"] = _normal(gen, (sum(need), page, hk, d), dt)
        s["table"] = table.cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["mask"] = None
        if not case["chain"]:
            # a node's parent is one of the nodes before it, or the context's last token
            parent = (torch.rand((r, n), generator=host) * (torch.arange(n) + 1)).long() - 1
            sees = torch.eye(n, dtype=torch.bool).expand(r, n, n).clone()
            for i in range(n):
                up = parent[:, i].clamp_min(0)
                sees[:, i] |= torch.gather(sees, 1, up[:, None, None].expand(r, 1, n))[:, 0] & (parent[:, i] >= 0)[:, None]
            words = (n + 63) // 64
            bits = torch.nn.functional.pad(sees, (0, 64 * words - n)).view(r, n, words, 64).long()
            s["mask"] = (bits << torch.arange(64)).sum(-1).cuda()
        s["scale"] = 1.0 / math.sqrt(d)
    return s


def _plain_conv(s):
    x, pool, slot, cu = s["x"], s["pool"], s["slot"].long(), s["cu"].long()
    c, w = s["weight"].shape
    n = slot.numel()
    rows = x.reshape(-1, c).float()
    kept = pool[slot].float()
    if s["has_state"] is not None:
        kept = torch.where((s["has_state"] != 0)[:, None, None], kept, torch.zeros_like(kept))
    ext = torch.cat([kept.reshape(n * (w - 1), c), rows])

    def source(first, at, seq):
        # row of ext that holds token `at` of the sequence `seq` that starts at token `first`
        return torch.where(at >= first, n * (w - 1) + at, seq * (w - 1) + (at - first) + (w - 1))

    t = torch.arange(rows.shape[0], device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    y = sum(ext[source(cu[seq], t - (w - 1) + j, seq)] * s["weight"][:, j] for j in range(w))
    if s["bias"] is not None:
        y = y + s["bias"]
    y = y / (1.0 + torch.exp(-y))
    nc = s["norm_channels"]
    if nc:
        h = y[:, :nc].reshape(-1, nc // 128, 128)
        h = h / torch.sqrt((h * h).sum(-1, keepdim=True) + s["eps"])
        y = torch.cat([h.reshape(-1, nc), y[:, nc:]], dim=1)
    i = torch.arange(w - 1, device=x.device)[None, :]
    seqs = torch.arange(n, device=x.device)[:, None]
    pool[slot] = ext[source(cu[:-1, None], cu[1:, None] - (w - 1) + i, seqs)].to(pool.dtype)
    return y.to(x.dtype).reshape(x.shape), pool


def _turn(x, cos, sin, interleaved):
    half = cos.shape[-1]
    body, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = body[..., 0::2], body[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)
    a, b = body[..., :half], body[..., half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)


def _plain_rope(s):
    angle = s["positions"].float()[:, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["scale"])[:, None], (torch.sin(angle) * s["scale"])[:, None]

    def one(x, weight):
        y = x.float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * weight
        return _turn(y, cos, sin, s["interleaved"]).to(x.dtype)

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if s["slots"] is None:
        return q, k
    s["k_cache"].flatten(0, 1)[s["slots"]] = k
    s["v_cache"].flatten(0, 1)[s["slots"]] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_tree(s):
    q, lens = s["q"], s["lens"].long()
    r, n, hq, d = q.shape
    hk = s["k_cache"].shape[2]
    table = s["table"].long()
    k = s["k_cache"][table].flatten(1, 2).permute(0, 2, 3, 1).float()   # [r, hk, d, l]
    v = s["v_cache"][table].flatten(1, 2).permute(0, 2, 1, 3).float()   # [r, hk, l, d]
    length = k.shape[-1]
    at = torch.arange(length, device=q.device)[None, None, :] - lens[:, None, None]   # node of a key, < 0: context
    i = torch.arange(n, device=q.device)[None, :, None]
    if s["mask"] is None:
        sees = at <= i
    else:
        word = torch.gather(s["mask"], 2, (at.clamp(0, n - 1) >> 6).expand(r, n, length))
        sees = (at < 0) | ((at < n) & ((word >> (at.clamp_min(0) & 63)) & 1).bool())
    rows = q.float().reshape(r, n, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(r, hk, -1, d)
    score = (rows @ k).reshape(r, hk, n, hq // hk, length) * s["scale"]
    score = torch.where(sees[:, None, :, None, :], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = (p.reshape(r, hk, -1, length) @ v).reshape(r, hk, n, hq // hk, d)
    out = out / torch.where(total > 0, total, torch.ones_like(total))
    return out.permute(0, 2, 1, 3, 4).reshape(r, n, hq, d).to(q.dtype)


def run(state):
    s = state
    if not own:
        return {"conv": _plain_conv, "rope": _plain_rope, "tree": _plain_tree}[s["op"]](s)
    import kda_chunked_prefill_02_gb300 as kda
    if s["op"] == "conv":
        y = kda.kda_short_conv(s["x"], s["weight"], bias=s["bias"], conv_state=s["pool"], slot=s["slot"],
                               has_state=s["has_state"], cu_seqlens=s["cu"] if s["packed"] else None,
                               norm_channels=s["norm_channels"], norm_eps=s["eps"])
        return y, s["pool"]
    if s["op"] == "rope":
        q, k = kda.kda_qk_norm_rope(s["q"], s["k"], s["positions"], s["freq"], q_weight=s["q_weight"],
                                    k_weight=s["k_weight"], norm_eps=s["eps"], interleaved=s["interleaved"],
                                    rope_scale=s["scale"], v=None if s["slots"] is None else s["v"],
                                    k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"])
        return (q, k) if s["slots"] is None else (q, s["k_cache"], s["v_cache"])
    return kda.kda_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], tree_mask=s["mask"],
                                  scale=s["scale"])


def work(case):
    if case["op"] == "conv":
        c, w, n = 3 * case["heads"] * 128, case["width"], case["requests"]
        t = case["tokens"] * (1 if case["form"] == "packed" else n)
        states = n + (n if case["form"] == "token" else sum(1 for i in range(n) if i % 3 != 1))
        return {"bytes": 4 * t * c + 2 * states * (w - 1) * c + 4 * c * (w + (1 if case["bias"] else 0)),
                "flops": t * c * (2 * w + 4 + (4 if case["norm"] else 0))}
    if case["op"] == "rope":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["k_heads"], case["dim"]
        heads = hq + (2 if case["cache"] else 1) * hk
        return {"bytes": 4 * t * heads * d + (12 if case["cache"] else 4) * t + 8 * d + 2 * case["rot"],
                "flops": t * (hq + hk) * (4 * d + 3 * case["rot"])}
    r, n, hq, hk, d = (case[x] for x in ("requests", "nodes", "q_heads", "k_heads", "dim"))
    lens = _lengths(r, case["context"])
    keys = sum(lens) + r * n
    words = 0 if case["chain"] else 8 * r * n * ((n + 63) // 64)
    return {"bytes": 4 * keys * hk * d + 4 * r * n * hq * d + words + 4 * r + 4 * sum((x + n + case["page"] - 1) // case["page"] for x in lens),
            "flops": 4 * hq * d * n * (sum(lens) + r)}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "conv":
        c, w = s["weight"].shape
        x = s["x"].reshape(-1, c)
        y = torch.empty(x.shape, dtype=f64, device=x.device)
        pool = s["pool"].to(f64)
        cu, slot = s["cu"].tolist(), s["slot"].tolist()
        kept = [1] * len(slot) if s["has_state"] is None else s["has_state"].tolist()
        for i, p in enumerate(slot):
            piece = torch.cat([pool[p] * kept[i], x[cu[i]:cu[i + 1]].to(f64)])
            length = cu[i + 1] - cu[i]
            z = torch.zeros((length, c), dtype=f64, device=x.device) + (0.0 if s["bias"] is None else s["bias"].to(f64))
            for j in range(w):
                z.addcmul_(piece[j:j + length], s["weight"][:, j].to(f64).expand(length, c))
            z = z * torch.sigmoid(z)
            for a in range(0, s["norm_channels"], 128):
                z[:, a:a + 128] *= torch.rsqrt(z[:, a:a + 128].square().sum(1, keepdim=True) + s["eps"])
            y[cu[i]:cu[i + 1]] = z
            pool[p] = piece[length:]
        return y.reshape(s["x"].shape), pool
    if case["op"] == "rope":
        angle = torch.outer(s["positions"].to(f64), s["freq"].to(f64))
        turn = torch.polar(torch.full_like(angle, s["scale"]), angle)[:, None]
        half = angle.shape[1]

        def one(x, weight):
            y = x.to(f64)
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * weight.to(f64)
            first, second = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["interleaved"]
                             else (slice(0, half), slice(half, 2 * half)))
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
        if s["slots"] is None:
            return q, k
        kc, vc = s["k_cache"].to(f64), s["v_cache"].to(f64)
        kc.flatten(0, 1)[s["slots"]] = k
        vc.flatten(0, 1)[s["slots"]] = s["v"].to(f64)
        return q, kc, vc
    r, n, hq, d = s["q"].shape
    hk, page = s["k_cache"].shape[2], s["k_cache"].shape[1]
    out = torch.empty(s["q"].shape, dtype=f64, device=s["q"].device)
    for i, length in enumerate(s["lens"].tolist()):
        pages = s["table"][i, :(length + n + page - 1) // page].long()
        k = s["k_cache"][pages].flatten(0, 1)[:length + n].to(f64).transpose(0, 1).repeat_interleave(hq // hk, 0)
        v = s["v_cache"][pages].flatten(0, 1)[:length + n].to(f64).transpose(0, 1).repeat_interleave(hq // hk, 0)
        sees = torch.ones((n, length + n), dtype=torch.bool, device=k.device)
        if s["mask"] is None:
            sees[:, length:] = torch.ones((n, n), dtype=torch.bool, device=k.device).tril()
        else:
            shift = torch.arange(64, device=k.device)
            sees[:, length:] = ((s["mask"][i][:, :, None] >> shift) & 1).bool().flatten(1)[:, :n]
        z = torch.matmul(s["q"][i].to(f64).transpose(0, 1), k.transpose(1, 2)) * s["scale"]
        p = torch.softmax(z.masked_fill(~sees, -math.inf), -1)
        out[i] = torch.matmul(p, v).transpose(0, 1)
    return out

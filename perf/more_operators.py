"""What a serving decoder runs between its KDA and attention operators: cases, inputs, plain forms.

Four operators:

* chunk: attention of chunks of new tokens (prompts, pieces of prompts, single
  tokens among them) over a paged cache;
* norm: a block's output added to the residual stream (with its own norm, a gate and
  a scale) and the norm in front of the next block;
* commit: the cache rows of a verified tree's accepted nodes moved together behind
  their context, in the caches of all layers;
* copy: entries of pools (cache pages, KDA states, convolution states of all layers)
  copied to others, for requests that are forked.

With `own` false, run() computes them with elementary torch operations in 32
bits; with `own` true it calls this repository's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # A few tokens behind a short context of one request: the latency of a small call.
        {"name": "chunk_small_r1", "op": "chunk", "requests": 1, "tokens": 16, "singles": 0, "context": 1000,
         "q_heads": 8, "k_heads": 2, "dim": 128, "page": 64, "padded": False, "dtype": "bf16"},
        # A whole prompt of one request.
        {"name": "chunk_prompt_t8192", "op": "chunk", "requests": 1, "tokens": 8192, "singles": 0, "context": 0,
         "q_heads": 32, "k_heads": 8, "dim": 128, "page": 64, "padded": False, "dtype": "bf16"},
        # A serving step that mixes 60 requests' next tokens with pieces of four prompts.
        {"name": "chunk_mixed_r64", "op": "chunk", "requests": 64, "tokens": 2108, "singles": 60, "context": 4096,
         "q_heads": 32, "k_heads": 8, "dim": 128, "page": 64, "padded": False, "dtype": "bf16"},
        # A piece of a very long prompt, far from its begin.
        {"name": "chunk_long_t2048", "op": "chunk", "requests": 1, "tokens": 2048, "singles": 0, "context": 126976,
         "q_heads": 32, "k_heads": 8, "dim": 128, "page": 64, "padded": False, "dtype": "bf16"},
        # Ragged prompts of odd lengths, one query head a key head, small pages, fp16.
        {"name": "chunk_ragged_r24", "op": "chunk", "requests": 24, "tokens": 12011, "singles": 1, "context": 700,
         "q_heads": 16, "k_heads": 16, "dim": 64, "page": 16, "padded": False, "dtype": "fp16"},
        # One token through one block: latency.
        {"name": "norm_token_t1", "op": "norm", "tokens": 1, "width": 2048, "post": False, "gate": "none",
         "residual": "bf16", "dtype": "bf16"},
        # A batch of prompts through a wide block with a norm behind it and an elementwise gate.
        {"name": "norm_prompts_t32768", "op": "norm", "tokens": 32768, "width": 4096, "post": True, "gate": "sigmoid",
         "residual": "bf16", "dtype": "bf16"},
        # An odd number of tokens, an odd width, the residual stream in fp32.
        {"name": "norm_odd_t8191", "op": "norm", "tokens": 8191, "width": 1288, "post": False, "gate": "plain",
         "residual": "fp32", "dtype": "fp16"},
        # One request's accepted path in a small model: latency.
        {"name": "commit_r1", "op": "commit", "requests": 1, "nodes": 8, "context": 300, "caches": 4, "heads": 2,
         "dim": 128, "page": 16, "dtype": "bf16"},
        # 256 requests' accepted paths of trees of 16 nodes in 16 layers.
        {"name": "commit_r256", "op": "commit", "requests": 256, "nodes": 16, "context": 100, "caches": 32, "heads": 8,
         "dim": 128, "page": 16, "dtype": "bf16"},
        # 24 forked requests' last pages, partly filled, in 16 layers.
        {"name": "copy_pages_n24", "op": "copy", "copies": 24, "entries": 64, "pools": 32, "rows": 64, "row": 1024,
         "partial": True, "dtype": "bf16"},
        # 16 forked requests' KDA states (32 heads of 128 x 128) in 12 layers.
        {"name": "copy_states_n16", "op": "copy", "copies": 16, "entries": 40, "pools": 12, "rows": 32, "row": 16384,
         "partial": False, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "norm", "commit", "copy"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "chunk":
        q_heads, k_heads, dim = rng.choice([(8, 2, 128), (32, 8, 128), (16, 16, 64), (32, 4, 128), (40, 8, 128),
                                            (16, 2, 256), (12, 4, 64), (64, 1, 128)])
        padded = rng.random() < 0.25
        requests = _log_int(rng, 1, 128)
        room = 16384 * min(1, 32 / q_heads)
        tokens = _log_int(rng, 1, max(1, int(room / requests if padded else room)))
        if not padded:
            tokens = max(tokens, requests)
        case = {"op": op, "requests": requests, "tokens": tokens,
                "singles": 0 if padded else rng.choice([0, 0, requests // 2, requests - 1]), "q_heads": q_heads,
                "k_heads": k_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128, 24]), "padded": padded,
                "dtype": dtype}
        new = _new_tokens(case)
        # no more scores than the largest listed case forms, all in all and for a key head of one request, and no
        # more keys than fit a cache of some GB
        most = min(2048 * 32 * 128 * 126976 // (sum(new) * q_heads * dim), 262144 * 8 * 128 // (requests * k_heads * dim),
                   2048 * 4 * 131072 // (max(new) * (q_heads // k_heads)), 131072) - max(new)
        case["context"] = 0 if most < 1 or rng.random() < 0.2 else _log_int(rng, 1, most)
        return case
    if op == "norm":
        width = 8 * _log_int(rng, 16, 1024)
        return {"op": op, "tokens": _log_int(rng, 1, 32768 * 4096 // 2 // width), "width": width,
                "post": rng.random() < 0.5, "gate": rng.choice(["none", "plain", "sigmoid"]),
                "residual": rng.choice([dtype, dtype, "fp32"]), "dtype": dtype}
    if op == "commit":
        requests, nodes = _log_int(rng, 1, 256), rng.choice([2, 4, 5, 8, 16, 31, 64])
        heads, dim = rng.choice([(2, 128), (8, 128), (4, 64), (1, 256), (3, 64)])
        return {"op": op, "requests": requests, "nodes": nodes, "context": rng.choice([1, 63, 100, 300]),
                "caches": 2 * _log_int(rng, 1, max(1, min(16, 256 * 400 * 32 * 1024 // (requests * (300 + nodes) * heads * dim) // 2))),
                "heads": heads, "dim": dim, "page": rng.choice([16, 64, 24]), "dtype": dtype}
    dtype = rng.choice(["bf16", "fp32"])
    rows, row = rng.choice([(16, 1024), (64, 1024), (24, 512), (3, 1536), (32, 16384), (10, 16384)])
    copies = _log_int(rng, 1, 64)
    entries = 2 * copies + rng.randrange(4)
    size = rows * row * (2 if dtype == "bf16" else 4)
    return {"op": op, "copies": copies, "entries": entries,
            "pools": _log_int(rng, 1, max(1, min(48, 12 * 16 * 2 * 1024 * 1024 // (copies * size)))), "rows": rows,
            "row": row, "partial": rng.random() < 0.5, "dtype": dtype}


def _contexts(requests, most):
    """Ragged context lengths, the first the longest: a fixed function of the case."""
    return [int(most * (1.0 if r == 0 else 0.2 + 0.8 * ((r * 0.6180339887) % 1.0))) for r in range(requests)]


def _new_tokens(case):
    """Every request's number of new tokens: `singles` of one, the others uneven."""
    n, t = case["requests"], case["tokens"]
    if case["padded"]:
        return [t] * n
    many = n - case["singles"]
    if many == 0:
        many = 1
    left = t - (n - many)
    weight = [0.15 + (r * 0.6180339887) % 1.0 for r in range(many)]
    take = [1 + int((left - many) * w / sum(weight)) for w in weight]
    take[0] += left - sum(take)
    return [1] * (n - many) + take


def _normal(gen, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if scale != 1.0 else dtype)
    return x if scale == 1.0 else (x * scale).to(dtype)


def _pages(lens, page, host):
    """A page table for the given lengths, the pages in a random order, and their number."""
    need = [max(1, (x + page - 1) // page) for x in lens]
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32)
    used = torch.arange(max(need))[None, :] < torch.tensor(need)[:, None]
    table[used] = torch.randperm(sum(need), generator=host).to(torch.int32)
    return table.cuda(), sum(need)


def _moved(case):
    """Every request's accepted path: ascending nodes of its tree, a fixed function of the case."""
    paths = []
    for r in range(case["requests"]):
        path, node = [], 0
        while node < case["nodes"]:
            if not path or (node * 7 + r * 3) % 5 < 3:
                path.append(node)
            node += 1 + (node + r) % 2
        paths.append(path[:max(1, len(path) - r % 3)])
    return paths


def _partial_rows(case):
    return [1 + (i * 29 + 11) % case["rows"] if case["partial"] else case["rows"] for i in range(case["copies"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    host = torch.Generator().manual_seed(1000003 * seed + 29)
    dt = _DT[case["dtype"]]
    s = {"op": case["op"]}
    if case["op"] == "chunk":
        hq, hk, d, page = (case[x] for x in ("q_heads", "k_heads", "dim", "page"))
        ctx, new = _contexts(case["requests"], case["context"]), _new_tokens(case)
        s["table"], pages = _pages([a + b for a, b in zip(ctx, new)], page, host)
        shape = (case["requests"], case["tokens"], hq, d) if case["padded"] else (case["tokens"], hq, d)
        s["q"] = _normal(gen, shape, dt, 1.5)
        s["k_cache"] = _normal(gen, (pages, page, hk, d), dt)
        s["v_cache"] = _normal(gen, (pages, page, hk, d), dt)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32).cuda()
        s["cu"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
        s["ctx_host"], s["new_host"] = ctx, new       # a scheduler that cuts prompts has made these lengths
        s["padded"] = case["padded"]
        s["scale"] = 1.0 / math.sqrt(d)
    elif case["op"] == "norm":
        t, e = case["tokens"], case["width"]
        s["y"] = _normal(gen, (t, e), dt)
        s["x"] = _normal(gen, (t, e), _DT[case["residual"]], 3.0)
        s["gate"] = None if case["gate"] == "none" else _normal(gen, (t, e), dt)
        s["sigmoid"] = case["gate"] == "sigmoid"
        s["post"] = 1.0 + _normal(gen, (e,), torch.float32, 0.1) if case["post"] else None
        s["weight"] = 1.0 + _normal(gen, (e,), torch.float32, 0.1)
        s["alpha"], s["eps"] = 0.75, 1e-6
    elif case["op"] == "commit":
        paths = _moved(case)
        ctx = [max(1, x) for x in _contexts(case["requests"], case["context"])]
        s["table"], pages = _pages([x + case["nodes"] for x in ctx], case["page"], host)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32).cuda()
        s["path"] = torch.tensor([p + [0] * (case["nodes"] - len(p)) for p in paths], dtype=torch.int32).cuda()
        s["accepted"] = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
        shape = (pages, case["page"], case["heads"], case["dim"])
        s["caches"] = [_normal(gen, shape, dt) for _ in range(case["caches"])]
    else:
        order = torch.randperm(case["entries"], generator=host).to(torch.int32)
        s["src"], s["dst"] = order[:case["copies"]].cuda(), order[case["copies"]:2 * case["copies"]].cuda()
        s["rows"] = torch.tensor(_partial_rows(case), dtype=torch.int32).cuda() if case["partial"] else None
        shape = (case["entries"], case["rows"], case["row"])
        s["pools"] = [_normal(gen, shape, dt) for _ in range(case["pools"])]
    return s


def _plain_chunk(s):
    q = s["q"].flatten(0, 1) if s["padded"] else s["q"]
    t, hq, d = q.shape
    page, hk = s["k_cache"].shape[1:3]
    g = hq // hk
    out = torch.empty_like(q)
    start = 0
    for r, (ctx, n) in enumerate(zip(s["ctx_host"], s["new_host"])):
        length = ctx + n
        pages = s["table"][r, :(length + page - 1) // page].long()
        k = s["k_cache"][pages].flatten(0, 1)[:length].permute(1, 2, 0).float()   # [hk, d, l]
        v = s["v_cache"][pages].flatten(0, 1)[:length].permute(1, 0, 2).float()   # [hk, l, d]
        rows = q[start:start + n].float().reshape(n, hk, g, d).permute(1, 0, 2, 3).reshape(hk, n * g, d)
        i = torch.arange(n, device=q.device).repeat_interleave(g)
        hidden = torch.arange(length, device=q.device)[None, :] > ctx + i[:, None]
        step = max(1, min(hk, (1 << 30) // (n * g * length)))
        parts = []
        for h in range(0, hk, step):
            score = rows[h:h + step] @ k[h:h + step]
            score.mul_(s["scale"]).masked_fill_(hidden, -math.inf)
            score.sub_(score.amax(-1, keepdim=True))
            score.exp_()
            total = score.sum(-1, keepdim=True)
            parts.append((score @ v[h:h + step]) / total)
            del score
        out[start:start + n] = torch.cat(parts).reshape(hk, n, g, d).permute(1, 0, 2, 3).reshape(n, hq, d).to(q.dtype)
        start += n
    return out.reshape(s["q"].shape)


def _plain_norm(s):
    u = s["y"].float()
    if s["post"] is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + s["eps"]) * s["post"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        u = u * (1.0 / (1.0 + torch.exp(-gate)) if s["sigmoid"] else gate)
    x = s["x"].float() + s["alpha"] * u
    h = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    return h.to(s["y"].dtype), x.to(s["x"].dtype)


def _plain_commit(s):
    n = s["path"].shape[1]
    page = s["caches"][0].shape[1]
    j = torch.arange(n, device=s["path"].device)[None, :].expand_as(s["path"])
    take = j < s["accepted"][:, None]
    request = torch.arange(s["path"].shape[0], device=j.device)[:, None].expand_as(j)[take]
    ctx = s["ctx"].long()[request]
    old, new = ctx + s["path"].long()[take], ctx + j[take]
    old_page, new_page = s["table"].long()[request, old // page], s["table"].long()[request, new // page]
    for cache in s["caches"]:
        cache[new_page, new % page] = cache[old_page, old % page]   # every row is read before one is written
    return s["caches"]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for pool in s["pools"]:
        if s["rows"] is None:
            pool[dst] = pool[src]
        else:
            take = torch.arange(pool.shape[1], device=pool.device)[None, :] < s["rows"][:, None]
            pool[dst] = torch.where(take[..., None], pool[src], pool[dst])
    return s["pools"]


def run(state):
    s = state
    if not own:
        return {"chunk": _plain_chunk, "norm": _plain_norm, "commit": _plain_commit, "copy": _plain_copy}[s["op"]](s)
    import kda_chunked_prefill_02_gb300 as kda
    if s["op"] == "chunk":
        return kda.kda_chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"],
                                       cu_seqlens=None if s["padded"] else s["cu"], scale=s["scale"],
                                       max_context=max(s["ctx_host"]))
    if s["op"] == "norm":
        return kda.kda_residual_norm(s["x"], s["y"], weight=s["weight"], post_norm=s["post"] is not None,
                                     post_weight=s["post"], gate=s["gate"], gate_sigmoid=s["sigmoid"],
                                     alpha=s["alpha"], norm_eps=s["eps"])
    if s["op"] == "commit":
        kda.kda_cache_commit(s["caches"], s["table"], s["ctx"], s["path"], s["accepted"])
        return s["caches"]
    kda.kda_pool_copy(s["pools"], s["src"], s["dst"], rows=s["rows"])
    return s["pools"]


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "chunk":
        hq, hk, d = case["q_heads"], case["k_heads"], case["dim"]
        ctx, new = _contexts(case["requests"], case["context"]), _new_tokens(case)
        keys = sum(ctx) + sum(new)
        return {"bytes": 4 * keys * hk * d + 4 * sum(new) * hq * d + 8 * case["requests"] + 4 * sum(
                    (a + b + case["page"] - 1) // case["page"] for a, b in zip(ctx, new)),
                "flops": 4 * hq * d * sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))}
    if case["op"] == "norm":
        t, e = case["tokens"], case["width"]
        stream = 4 if case["residual"] == "fp32" else 2
        return {"bytes": t * e * (4 + 2 * stream + (0 if case["gate"] == "none" else 2)) + 4 * e * (2 if case["post"] else 1),
                "flops": t * e * (6 + (4 if case["post"] else 0) + (0 if case["gate"] == "none" else 4))}
    if case["op"] == "commit":
        paths = _moved(case)
        moved = sum(1 for p in paths for j, node in enumerate(p) if node != j)
        return {"bytes": 2 * moved * case["caches"] * case["heads"] * case["dim"] * size + 4 * sum(map(len, paths)) + 8 * len(paths),
                "flops": 0}
    return {"bytes": 2 * sum(_partial_rows(case)) * case["row"] * size * case["pools"] + 8 * case["copies"], "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "chunk":
        q = s["q"].reshape(-1, *s["q"].shape[-2:])
        hk, page = case["k_heads"], case["page"]
        g = case["q_heads"] // hk
        if work(case)["flops"] > 9e12:
            return None
        out = torch.empty(q.shape, dtype=f64, device=q.device)
        cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
        for r, c in enumerate(ctx):
            a, b = cu[r], cu[r + 1]
            at = torch.arange(c + b - a, device=q.device)
            row = s["table"][r].long()[at // page], at % page
            for h in range(hk):
                k, v = s["k_cache"][row[0], row[1], h].to(f64), s["v_cache"][row[0], row[1], h].to(f64)
                block = max(1, (1 << 28) // (at.numel() * g))
                for i in range(a, b, block):
                    e = min(b, i + block)
                    z = torch.einsum("thd,ld->thl", q[i:e, h * g:(h + 1) * g].to(f64), k) * s["scale"]
                    late = at[None, :] > c + torch.arange(i - a, e - a, device=q.device)[:, None]
                    z.masked_fill_(late[:, None, :], -math.inf)
                    out[i:e, h * g:(h + 1) * g] = torch.einsum("thl,ld->thd", torch.softmax(z, -1), v)
        return out.reshape(s["q"].shape)
    if case["op"] == "norm":
        y, x = s["y"].to(f64), s["x"].to(f64)
        if s["post"] is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * s["post"].to(f64)
        if s["gate"] is not None:
            y = y * (torch.sigmoid(s["gate"].to(f64)) if s["sigmoid"] else s["gate"].to(f64))
        x = torch.add(x, y, alpha=s["alpha"])
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].to(f64), x
    if case["op"] == "commit":
        page, table = case["page"], s["table"].tolist()
        for r, (c, count) in enumerate(zip(s["ctx"].tolist(), s["accepted"].tolist())):
            nodes = s["path"][r, :count].tolist()
            place = [[], [], [], []]
            for j, node in enumerate(nodes):
                for at, p in ((0, c + node), (2, c + j)):
                    place[at].append(table[r][p // page])
                    place[at + 1].append(p % page)
            place = [torch.tensor(x, device="cuda") for x in place]
            for cache in s["caches"]:
                cache.index_put_((place[2], place[3]), cache[place[0], place[1]].clone())
        return s["caches"]
    rows = _partial_rows(case)
    for a, b, n in zip(s["src"].tolist(), s["dst"].tolist(), rows):
        for pool in s["pools"]:
            pool[b, :n].copy_(pool[a, :n])
    return s["pools"]

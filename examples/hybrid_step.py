"""One serving step of a small decoder that mixes KDA layers with softmax-attention
layers: a ragged batch of prompts, the verification of a tree of drafted tokens for
every request, the next token behind the accepted ones, and a request that is forked.

    python examples/hybrid_step.py

The model is a stack of pairs (a KDA layer, an attention layer) with random weights
and plain torch matrix products between the operators.  KDA layers run
kda_short_conv -> kda_prefill on the prompts and kda_short_conv -> kda_verify on the
drafts, where every root-to-leaf path of a tree is a request of kda_verify (a state
belongs to a path); attention layers run kda_qk_norm_rope, which puts keys and values
into the paged cache, -> kda_chunk_attention, one call for all prompts, or
kda_tree_attention, one call for all trees.  Between them kda_residual_norm adds a
layer's output to the residual stream and norms it for the next.  The accepted paths
are then committed: to the KDA layers' states, and by kda_cache_commit to the caches,
where they move together behind their context.  A fork is a kda_pool_copy of the
request's pages and states.  The step is checked against running the accepted paths
token by token.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_chunked_prefill_02_gb300 as K  # noqa: E402

H, D = 4, 128                     # KDA heads
HQ, HK = 8, 2                     # attention heads
E = H * D                         # model width
W, PAGE, LAYERS = 4, 16, 2
BF16 = torch.bfloat16


class Weights:
    def __init__(self, gen):
        def mat(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") / shape[0] ** 0.5).to(BF16)
        self.layers = []
        for _ in range(LAYERS):
            self.layers.append(dict(
                qkv=mat(E, 3 * E), gate=mat(E, E), beta=mat(E, H), out=mat(E, E),
                conv=torch.randn((3 * E, W), generator=gen, device="cuda") / W ** 0.5,
                aqkv=mat(E, (HQ + 2 * HK) * D), aout=mat(HQ * D, E),
                qw=torch.ones(D, device="cuda"), kw=torch.ones(D, device="cuda")))


def gates(x, w):
    """Log decays in (-5, 0) and beta logits of a KDA layer."""
    return -5.0 * torch.sigmoid((x @ w["gate"]).float()).unflatten(-1, (H, D)), (x @ w["beta"]).float()


class Decoder:
    def __init__(self, requests, room, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w = Weights(gen).layers
        self.gen, self.R = gen, requests
        pages = (room + PAGE - 1) // PAGE
        self.table = torch.randperm(requests * pages, device="cuda").to(torch.int32).view(requests, pages)
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.conv = [torch.zeros((requests, W - 1, 3 * E), dtype=BF16, device="cuda") for _ in self.w]
        self.state = [torch.zeros((requests, H, D, D), device="cuda") for _ in self.w]
        self.kc = [torch.zeros((requests * pages, PAGE, HK, D), dtype=BF16, device="cuda") for _ in self.w]
        self.vc = [torch.zeros_like(c) for c in self.kc]
        self.freq, self.scale = K.rope_frequencies(D, base=1e6, scaling="by_parts", factor=8.0, original_context=4096)

    def slots(self, request, position):
        return (self.table[request, position // PAGE].long() * PAGE + position % PAGE)

    def attention_in(self, w, i, x, positions, slots):
        """Queries of normed tokens x [T, E]; their keys and values go into the cache."""
        qkv = (x @ w["aqkv"]).view(-1, HQ + 2 * HK, D)
        q, _ = K.kda_qk_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HK], positions.to(torch.int32), self.freq,
                                  q_weight=w["qw"], k_weight=w["kw"], rope_scale=self.scale, v=qkv[:, HQ + HK:],
                                  k_cache=self.kc[i], v_cache=self.vc[i], slots=slots)
        return q

    def prompt(self, x, cu):
        """A packed batch of prompts x [T, E], request n's tokens cu[n] .. cu[n+1]-1."""
        lens = cu[1:] - cu[:-1]
        request = torch.repeat_interleave(torch.arange(self.R, device="cuda"), lens)
        position = torch.arange(x.shape[0], device="cuda") + (self.lens - cu[:-1]).long()[request]
        h, _ = K.kda_residual_norm(x)
        for i, w in enumerate(self.w):
            y = K.kda_short_conv(h @ w["qkv"], w["conv"], conv_state=self.conv[i], cu_seqlens=cu,
                                 norm_channels=2 * E).unflatten(-1, (3 * H, D))
            g, beta = gates(h, w)
            o, fin = K.kda_prefill(y[:, :H], y[:, H:2 * H], y[:, 2 * H:], g, beta, initial_state=self.state[i],
                                   cu_seqlens=cu)
            self.state[i].copy_(fin)
            h, x = K.kda_residual_norm(x, o.flatten(1) @ w["out"])
            q = self.attention_in(w, i, h, position, self.slots(request, position))
            a = K.kda_chunk_attention(q, self.kc[i], self.vc[i], self.table, self.lens, cu_seqlens=cu)
            h, x = K.kda_residual_norm(x, a.flatten(1) @ w["aout"])
        self.lens += lens
        return x

    def verify(self, x, parents, accepted=None):
        """Trees of N drafts a request, x [R, N, E], parents [R, N] on the host.  With
        `accepted` (a list of a path's nodes a request) the state after them is kept."""
        N = x.shape[1]
        mask = K.tree_mask(parents.cuda())
        paths, of = [], []                       # root-to-leaf paths, padded with their leaf
        for r in range(self.R):
            inner = set(parents[r].tolist())
            for leaf in (i for i in range(N) if i not in inner):
                p = [leaf]
                while int(parents[r, p[0]]) >= 0:
                    p.insert(0, int(parents[r, p[0]]))
                paths.append(p)
                of.append(r)
        depth = max(map(len, paths))
        of = torch.tensor(of, device="cuda")
        idx = torch.tensor([p + [p[-1]] * (depth - len(p)) for p in paths], device="cuda")
        level = torch.zeros(x.shape[:2], dtype=torch.int64)
        for r in range(self.R):
            for i in range(N):
                level[r, i] = level[r, parents[r, i]] + 1 if parents[r, i] >= 0 else 0
        position = self.lens[:, None] + level.cuda()
        row = self.lens[:, None].long() + torch.arange(N, device="cuda")        # a node's place in the cache
        slots = self.slots(torch.arange(self.R, device="cuda")[:, None], row).flatten().contiguous()
        zero = torch.zeros(len(paths), dtype=torch.int32, device="cuda")
        h, _ = K.kda_residual_norm(x)
        for i, w in enumerate(self.w):
            # the KDA layer runs every path from a copy of its request's states
            proj = (h @ w["qkv"])[of[:, None], idx]
            conv, state = self.conv[i][of].contiguous(), self.state[i][of].contiguous()
            y = K.kda_short_conv(proj, w["conv"], conv_state=conv, accepted=zero,
                                 norm_channels=2 * E).unflatten(-1, (3 * H, D))
            g, beta = gates(h, w)
            g, beta = g[of[:, None], idx].contiguous(), beta[of[:, None], idx].contiguous()
            o = K.kda_verify(y[:, :, :H], y[:, :, H:2 * H], y[:, :, 2 * H:], g, beta, state, zero)
            if accepted is not None:
                # commit: the request's own states, through its accepted path's drafts alone
                first = [next(j for j in range(len(paths)) if int(of[j]) == r and paths[j][:len(a)] == a)
                         for r, a in enumerate(accepted)]
                acc = torch.tensor([len(a) for a in accepted], dtype=torch.int32, device="cuda")
                K.kda_short_conv(proj[first], w["conv"], conv_state=self.conv[i], accepted=acc, state_only=True)
                yf = y[first]
                K.kda_verify(yf[:, :, :H], yf[:, :, H:2 * H], yf[:, :, 2 * H:], g[first], beta[first], self.state[i],
                             acc, replay_only=True)
            out = torch.empty((self.R, N, E), dtype=BF16, device="cuda")
            out[of[:, None], idx] = o.flatten(2)      # nodes that paths share: the same values
            h, x = K.kda_residual_norm(x, out @ w["out"])
            q = self.attention_in(w, i, h.flatten(0, 1), position.flatten().contiguous(), slots)
            a = K.kda_tree_attention(q.view(self.R, N, HQ, D), self.kc[i], self.vc[i], self.table, self.lens,
                                     tree_mask=mask)
            h, x = K.kda_residual_norm(x, a.flatten(2) @ w["aout"])
        if accepted is not None:
            path = torch.tensor([a + [0] * (N - len(a)) for a in accepted], dtype=torch.int32, device="cuda")
            count = torch.tensor([len(a) for a in accepted], dtype=torch.int32, device="cuda")
            K.kda_cache_commit(self.kc + self.vc, self.table, self.lens, path, count)
        return x

    def fork(self, parent, child):
        """Request `child` goes on from where `parent` is."""
        src, dst = torch.tensor([[parent], [child]], dtype=torch.int32, device="cuda")
        K.kda_pool_copy(self.state + self.conv, src, dst)
        K.kda_pool_copy(self.kc + self.vc, self.table[parent], self.table[child])   # (a server copies the last page)
        self.lens[child] = self.lens[parent]


def main():
    torch.manual_seed(0)
    lens = [37, 5, 18]
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2], [-1, 0, 1, 2, 0, 4], [-1, -1, 1, 1, 3, 0]])
    accepted = [[0, 1, 4], [0, 1, 2, 3], [1, 3]]
    R, N = parents.shape
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randn((sum(lens), E), generator=gen, device="cuda").to(BF16)
    drafts = torch.randn((R, N, E), generator=gen, device="cuda").to(BF16)

    tree = Decoder(R, 128)
    tree.prompt(prompts, cu)
    y = tree.verify(drafts, parents, accepted)

    # the accepted paths, one token after the other, as trees of one node
    step = Decoder(R, 128)
    step.prompt(prompts, cu)
    worst = 0.0
    for d in range(max(map(len, accepted))):
        node = [a[min(d, len(a) - 1)] for a in accepted]
        x = drafts[torch.arange(R), node][:, None]
        live = [d < len(a) for a in accepted]
        keep = [[0] if v else [] for v in live]
        z = step.verify(x, torch.full((R, 1), -1), keep)
        for r in range(R):
            if live[r]:
                worst = max(worst, float((z[r, 0].float() - y[r, node[r]].float()).abs().max()))
        step.lens += torch.tensor(live, dtype=torch.int32, device="cuda")
    # the next token behind what was accepted, and behind a fork of the first request
    tree.lens += torch.tensor([len(a) for a in accepted], dtype=torch.int32, device="cuda")
    state = max(float((a - b).norm() / a.norm()) for a, b in zip(tree.state, step.state))
    conv = all(torch.equal(a, b) for a, b in zip(tree.conv[:1], step.conv[:1]))
    size = float(y.float().abs().max())
    x, root = torch.randn((R, 1, E), generator=gen, device="cuda").to(BF16), torch.full((R, 1), -1)
    worst = max(worst, float((tree.verify(x, root).float() - step.verify(x, root).float()).abs().max()))
    tree.fork(0, 2)
    z = tree.verify(x[:1].expand(R, 1, E).contiguous(), root)
    worst = max(worst, float((z[0].float() - z[2].float()).abs().max()))
    print("tree step against token by token: outputs within %.3f (largest %.1f), KDA states within %.1e, first layer's "
          "conv states %s" % (worst, size, state, "equal" if conv else "differ"))
    return worst, size, state, conv


if __name__ == "__main__":
    main()

"""Speculative decoding of a toy model over the cache, with its streaming, on one GPU.

    PYTHONPATH=. python examples/speculative.py

A few random decoder layers with grouped query heads run from prompt to generated
tokens on the library's operators alone: every layer appends its new tokens to the
cache (rotary positions) and attends it; the prompts' rows go to a host replica. Each step
drafts a small tree of tokens per sequence from what followed the last token before,
checks the whole tree in one pass (tree attention), keeps the longest path that the
model itself would have taken, moves that path's rows together (compact) and appends
them to the replica. The tokens are those of one-token-at-a-time decoding.
"""
import numpy as np
import torch

import kv_cache_streaming_gb300 as dv

L, B, H, G, D, S, VOCAB = 3, 3, 2, 4, 64, 512, 96
DTYPE = torch.float16


class Model:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        d = H * G * D

        def w(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[0] ** -0.5).to(DTYPE)

        self.embed = torch.randn(VOCAB, d, generator=g, device="cuda").to(DTYPE)
        self.qkv = [w(d, (H * G + 2 * H) * D) for _ in range(L)]
        self.out = [w(d, d) for _ in range(L)]
        self.head = w(d, VOCAB)
        self.rope = dv.Rope(D, base=10000.0, scaling="parts", factor=4.0, original_max=S)
        self.k = torch.zeros(L * B * H * D * S, dtype=DTYPE, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.cache = dv.Cache(L, B, H, D, S, 2, self.k, self.v)

    def forward(self, tokens, s, e, tree=None, positions=None, prompt=False):
        """Logits of the packed new tokens, which take rows [s, e) of the cache."""
        x = self.embed[tokens]
        n, hq = len(tokens), H * G
        ws = torch.empty(max(1, dv.dv_attention_workspace(self.cache, s, e, hq)), dtype=torch.uint8, device="cuda")
        for l in range(L):
            h = torch.nn.functional.layer_norm(x.float(), x.shape[1:]).to(DTYPE) @ self.qkv[l]
            q, k, v = (t.view(n, -1, D) for t in h.split([hq * D, H * D, H * D], dim=1))  # strided rows
            q = dv.dv_kv_append(self.cache, l, s, e, k, v, q=q, rope=self.rope, positions=positions)
            o = torch.empty(n, hq, D, dtype=DTYPE, device="cuda")
            if prompt:
                dv.dv_prompt_attention(self.cache, l, s, e, q, o, D ** -0.5, ws)
            else:
                dv.dv_tree_attention(self.cache, l, s, e, q, o, D ** -0.5, ws, tree=tree)
            x = x + o.view(n, -1) @ self.out[l]
        return torch.nn.functional.layer_norm(x.float(), x.shape[1:]) @ self.head.float()


def draft_tree(root, follows, limit=16):
    """(tokens, parents) of a tree below the last token: up to two continuations a
    node, among the tokens that followed it so far."""
    tokens, parents = [root], [-1]
    for i in range(limit):
        if i == len(tokens):
            break
        for t in list(follows.get(tokens[i], ()))[-2:]:
            if len(tokens) < limit:
                tokens.append(t)
                parents.append(i)
    return tokens, parents


def generate(prompts, steps, speculative, model=None):
    """Greedy tokens after each prompt; the model (with its cache) and the replica."""
    m = model or Model()
    zero, e = np.zeros(B, np.int32), np.array([len(p) for p in prompts], np.int32)
    arena = dv.host_empty(2 * L * B * H * D * S * 2)
    rep = dv.Replica(arena, B)
    logits = m.forward(torch.tensor(sum(prompts, []), device="cuda"), zero, e, prompt=True)
    rep.append(m.cache, 0, L, zero, e, step=0)  # the prompts' rows, to the host
    nxt = logits[torch.from_numpy(np.cumsum(e) - 1).cuda()].argmax(-1).tolist()
    got = [[t] for t in nxt]
    follows = [{} for _ in range(B)]
    for b, p in enumerate(prompts):
        for a, z in zip(p + nxt[b:b + 1], (p + nxt[b:b + 1])[1:]):
            follows[b].setdefault(a, {})[z] = True
    lens, step, drafted = e.copy(), 0, 0
    while min(len(g) for g in got) < steps:
        step += 1
        trees = [draft_tree(g[-1], f) if speculative else ([g[-1]], [-1]) for g, f in zip(got, follows)]
        n = np.array([len(t) for t, _ in trees], np.int32)
        depth, bits = [], []
        for t, parents in trees:
            d, a = [], []
            for i, p in enumerate(parents):
                d.append(d[p] + 1 if i else 0)
                a.append((a[p] if i else 0) | 1 << i)
            depth.append(d)
            bits += a
        at = np.concatenate([ln + np.array(d, np.int32) for ln, d in zip(lens, depth)]).astype(np.int32)
        logits = m.forward(torch.tensor(sum((t for t, _ in trees), []), device="cuda"), lens, lens + n,
                           tree=torch.tensor(bits, device="cuda"), positions=torch.from_numpy(at).cuda())
        best = logits.argmax(-1).tolist()
        keep, kept, base = [], [], 0
        for b, (t, parents) in enumerate(trees):
            path = [0]
            while True:  # down the tree, along what the model itself picks
                pick = best[base + path[-1]]
                down = [i for i in range(len(t)) if parents[i] == path[-1] and t[i] == pick]
                follows[b].setdefault(t[path[-1]], {}).pop(pick, None)
                follows[b][t[path[-1]]][pick] = True
                got[b].append(pick)
                if not down:
                    break
                path.append(down[0])
            base += len(t)
            keep += [lens[b] + i for i in path]
            kept.append(len(path))
        drafted += sum(kept)
        end = lens + np.array(kept, np.int32)
        dv.dv_kv_compact(m.cache, 0, L, lens, end, torch.tensor(keep, dtype=torch.int32, device="cuda"))
        rep.append(m.cache, 0, L, lens, end, step=step)  # the accepted rows, to the host
        lens = end
    torch.cuda.synchronize()
    return {"tokens": [g[:steps] for g in got], "model": m, "replica": rep, "arena": arena, "lens": lens,
            "steps": step, "rows": drafted}


def main(steps=40):
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (37, 5, 140)]
    return prompts, generate(prompts, steps, True), generate(prompts, steps, False)


if __name__ == "__main__":
    _, spec, plain = main()
    assert spec["tokens"] == plain["tokens"]
    print(f"the same {sum(map(len, plain['tokens']))} tokens in {spec['steps']} passes instead of {plain['steps']}")

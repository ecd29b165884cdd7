"""Measured cases of the operators over the KV cache: appending new tokens with rotary positions, causal attention of
packed prompts, attention of drafted token trees (one token: a decode step), and compacting cache rows in place.

Cache layout of one layer, with 8 elements of 2 bytes per 16-byte chunk: K [B][H][D/8][S][8], V [B][H][S][D].
A case's ragged lengths come from its own number `ranges`; its values come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---- cases --------------------------------------------------------------------------------------------------------

def listed():
    gpt2 = dict(dtype="fp16", B=8, H=25, G=1, D=64, S=1024)
    opt = dict(dtype="fp16", B=8, H=40, G=1, D=128, S=2048)
    bloom = dict(dtype="bf16", B=32, H=112, G=1, D=128, S=2048)
    grouped = dict(dtype="bf16", H=8, G=8, D=128)
    rope = dict(layout="half", rot=64, base=10000.0, scaling="none", factor=1.0, original=0)
    return [
        # one decode token of 8 short sequences: latency of the smallest append
        dict(name="append_one_token", op="append", **gpt2, ctx=500, ctx_hi=1000, new=1, new_hi=1, tree=False,
             **rope, ranges=1),
        # ragged prompts written at once; half of the head rotated, interleaved pairs
        dict(name="append_prompts", op="append", **opt, ctx=0, ctx_hi=0, new=16, new_hi=2048, tree=False,
             layout="interleaved", rot=64, base=10000.0, scaling="none", factor=1.0, original=0, ranges=2),
        # trees of drafted tokens far into a long context, frequencies scaled by parts, grouped heads
        dict(name="append_tree_far", op="append", **grouped, B=4, S=131072, ctx=60000, ctx_hi=131000, new=17, new_hi=64,
             tree=True, layout="half", rot=128, base=500000.0, scaling="parts", factor=16.0, original=8192, ranges=3),
        # eight prompts of 1000 tokens, small heads
        dict(name="prompt_equal", op="prompt", **gpt2, ctx=0, ctx_hi=0, new=1000, new_hi=1000, ranges=4),
        # a full batch of ragged prompts, many heads
        dict(name="prompt_ragged", op="prompt", **bloom, ctx=0, ctx_hi=0, new=64, new_hi=1536, ranges=5),
        # a chunk of a long prompt after an earlier part, grouped heads
        dict(name="prompt_chunk_long", op="prompt", **grouped, B=1, S=32768, ctx=28672, ctx_hi=28672, new=4096,
             new_hi=4096, ranges=6),
        # one decode token over short contexts: latency
        dict(name="decode_short", op="tree", **gpt2, ctx=100, ctx_hi=1000, new=1, new_hi=1, tree=False, ranges=7),
        # drafted trees of different sizes over ragged contexts
        dict(name="tree_ragged", op="tree", **opt, ctx=16, ctx_hi=1980, new=5, new_hi=33, tree=True, ranges=8),
        # one decode token of a full batch, many heads
        dict(name="decode_batch", op="tree", **bloom, ctx=64, ctx_hi=1791, new=1, new_hi=1, tree=False, ranges=9),
        # wide trees over long contexts, grouped heads
        dict(name="tree_long_grouped", op="tree", **grouped, B=2, S=131072, ctx=100000, ctx_hi=131000, new=64, new_hi=64,
             tree=True, ranges=10),
        # the accepted path of each tree moved to the front of its tree, in every layer
        dict(name="compact_accepted", op="compact", **opt, L=8, ctx=16, ctx_hi=1980, new=4, new_hi=8, far=False,
             ranges=11),
        # the first rows kept and a recent window moved down behind them
        dict(name="compact_window", op="compact", **gpt2, L=24, ctx=4, ctx_hi=4, new=300, new_hi=509, far=True,
             ranges=12),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "prompt", "tree", "compact"])
    G = rng.choice([1, 1, 2, 4, 5, 8])
    D = rng.choice([64, 128, 64, 128, 80, 96])
    case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), B=spread(1, 32), H=spread(1, 40), G=G, D=D,
                ranges=rng.randrange(1 << 30))
    if op == "prompt":
        top = spread(1, 8192)
        # keeps sequences x heads x length^2 below the largest listed case
        while case["B"] * case["H"] * G * top * top > 64 * 4096 * 8192:
            case["B"] = max(1, case["B"] // 2)
            top = max(1, top // 2) if case["B"] == 1 else top
        ctx = rng.choice([0, 0, spread(1, 4096)])
        while case["B"] * case["H"] * G * top * (top + ctx) > 64 * 4096 * 16384 and ctx:
            ctx //= 2
        case |= dict(ctx=ctx // 2, ctx_hi=ctx, new=max(1, top // rng.choice([1, 2, 8])), new_hi=top,
                     S=ctx + top + rng.randrange(0, 70))
    elif op == "compact":
        n = spread(1, 400)
        far = n > 16 or rng.random() < 0.5
        case |= dict(L=spread(1, 12), ctx=rng.randrange(0, 9), ctx_hi=rng.choice([9, 300]), new=max(1, n // 2), new_hi=n,
                     far=far)
        case["S"] = case["ctx_hi"] + (2 * n if far else n + 40) + rng.randrange(1, 70)
    else:
        n = rng.choice([1, 1, spread(1, 64)])
        if op == "append" and rng.random() < 0.5:
            n = spread(1, 2048)
        ctx = spread(1, 32768)
        while case["B"] * case["H"] * D * (ctx + n) > (1 << 28):
            case["B"], ctx = max(1, case["B"] // 2), max(1, ctx // 2)
        case |= dict(ctx=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx, new=max(1, n // rng.choice([1, 2])), new_hi=n,
                     S=ctx + n + rng.randrange(0, 70), tree=1 < n <= 64 and rng.random() < 0.7)
        if op == "append":
            case |= dict(layout=rng.choice(["half", "interleaved"]), rot=rng.choice([D, D // 2, 32]),
                         base=rng.choice([10000.0, 500000.0]), scaling=rng.choice(["none", "linear", "ntk", "parts"]),
                         factor=rng.choice([2.0, 4.0, 16.0]), original=rng.choice([2048, 4096, 8192]))
    return case


def lengths(case):
    """Rows before the new ones and new rows of each sequence, int32 arrays."""
    r = random.Random(case["ranges"])
    ctx = [r.randint(case["ctx"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [r.randint(case["new"], case["new_hi"]) for _ in range(case["B"])]
    return np.array(ctx, np.int32), np.array(new, np.int32)


def work(case):
    s, n = lengths(case)
    s, n = s.astype(np.int64), n.astype(np.int64)
    H, D, Hq, T = case["H"], case["D"], case["H"] * case["G"], int(n.sum())
    if case["op"] == "append":
        return {"bytes": 2 * 2 * T * (Hq + 2 * H) * D + (4 * T if case["tree"] else 0), "flops": 3 * T * (Hq + H) * case["rot"]}
    if case["op"] == "compact":
        keep = keep_rows(case)
        moved = sum(int((k != np.arange(a, a + len(k))).sum()) for k, a in zip(keep, s))
        return {"bytes": 2 * 2 * 2 * case["L"] * H * D * moved + 4 * T, "flops": 0}
    rows = int((s + n).sum())
    if case["op"] == "tree" and case["tree"]:
        bits, _ = trees(case)
        pairs = int((s * n).sum()) + sum(int(b).bit_count() for b in bits)
    else:
        pairs = int((s * n + n * (n + 1) // 2).sum())
    return {"bytes": 2 * (2 * T * Hq * D + 2 * rows * H * D) + (8 * T if case.get("tree") else 0),
            "flops": 4 * D * Hq * pairs}


def trees(case):
    """Ancestor bits (itself included) and depth of each drafted node; parents come before their children."""
    r = random.Random(case["ranges"] + 1)
    bits, depth = [], []
    for n in lengths(case)[1]:
        b, d = [], []
        for i in range(int(n)):
            p = r.randint(max(0, (i - 1) // 4), i - 1) if i else -1
            b.append((b[p] if i else 0) | 1 << i)
            d.append(d[p] + 1 if i else 0)
        bits += b
        depth += d
    return bits, depth


def keep_rows(case):
    """The row each destination row is filled from: `far`, the last rows in use; else the path of a tree of up to 32
    more nodes (its first node is in place, the others come after the rows that are kept)."""
    r = random.Random(case["ranges"] + 2)
    s, n = lengths(case)
    out = []
    for a, k in zip(s.tolist(), n.tolist()):
        if case["far"]:
            out.append(np.arange(a + k, a + 2 * k, dtype=np.int32))
        else:
            path = [a] + sorted(r.sample(range(a + k, a + k + 32), k - 1)) if k <= 32 else list(range(a, a + k))
            out.append(np.array(path, np.int32))
    return out


# ---- inputs -------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, B, H, D, S = DTYPES[case["dtype"]], case["B"], case["H"], case["D"], case["S"]
    Hq, L = H * case["G"], case.get("L", 1)
    s, n = lengths(case)
    T = int(n.sum())

    def normal(*shape):
        return torch.empty(*shape, dtype=dt, device="cuda").normal_(generator=g)

    st = dict(case=case, s=s, e=s + n, k=normal(L, B, H, D // 8, S, 8), v=normal(L, B, H, S, D))
    if case["op"] == "append":
        # one fused projection's rows: queries, keys, values side by side
        qkv = normal(T, (Hq + 2 * H) * D)
        st |= dict(qn=qkv[:, :Hq * D].view(T, Hq, D), kn=qkv[:, Hq * D:(Hq + H) * D].view(T, H, D),
                   vn=qkv[:, (Hq + H) * D:].view(T, H, D), q_out=torch.empty(T, Hq, D, dtype=dt, device="cuda"))
        st["positions"] = None
        if case["tree"]:
            at = np.repeat(s, n) + np.array(trees(case)[1], np.int32)
            st["positions"] = torch.from_numpy(at.astype(np.int32)).cuda()
    elif case["op"] == "compact":
        st["keep"] = torch.from_numpy(np.concatenate(keep_rows(case))).cuda()
    else:
        st |= dict(q=normal(T, Hq, D) * 2, out=torch.empty(T, Hq, D, dtype=dt, device="cuda"), scale=D ** -0.5, bits=None)
        if case["op"] == "tree" and case["tree"]:
            bits = np.array(trees(case)[0], np.uint64).view(np.int64)
            st["bits"] = torch.from_numpy(bits).cuda()
    if own:  # what a program keeps between its calls: the cache's description, the rotation, the workspace
        import kv_cache_streaming_gb300 as dv
        st["cache"] = dv.Cache(L, B, H, D, S, 2, st["k"], st["v"])
        if case["op"] == "append":
            st["rope"] = dv.Rope(case["rot"], interleaved=case["layout"] == "interleaved", base=case["base"],
                                 scaling=case["scaling"], factor=case["factor"], original_max=case["original"])
        elif case["op"] != "compact":
            st["workspace"] = torch.empty(dv.dv_attention_workspace(st["cache"], s, s + n, Hq), dtype=torch.uint8,
                                          device="cuda")
    return st


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        import kv_cache_streaming_gb300 as dv
        c, s, e = st["cache"], st["s"], st["e"]
        if op == "append":
            dv.dv_kv_append(c, 0, s, e, st["kn"], st["vn"], q=st["qn"], q_out=st["q_out"], rope=st["rope"],
                            positions=st["positions"])
            return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
        if op == "compact":
            dv.dv_kv_compact(c, 0, st["k"].shape[0], s, e, st["keep"])
            return {"k": st["k"].view(torch.int16), "v": st["v"].view(torch.int16)}
        if op == "prompt":
            dv.dv_prompt_attention(c, 0, s, e, st["q"], st["out"], st["scale"], st["workspace"])
        else:
            dv.dv_tree_attention(c, 0, s, e, st["q"], st["out"], st["scale"], st["workspace"], tree=st["bits"])
        return st["out"]
    return {"append": plain_append, "compact": plain_compact}.get(op, plain_attention)(st)


def frequencies(case):
    """Angle per position of each rotated pair, and the factor on the rotated values (float64, on the host)."""
    rot, base, kind, f = case["rot"], case["base"], case["scaling"], case["factor"]
    i = np.arange(rot // 2, dtype=np.float64)
    if kind == "ntk":
        base = base * f ** (rot / (rot - 2))
    inv = base ** (-2 * i / rot)
    if kind == "linear":
        inv = inv / f
    if kind == "parts":
        turns = case["original"] * inv / (2 * math.pi)
        fast = np.clip((turns - 1) / (32 - 1), 0, 1)
        return inv * fast + inv / f * (1 - fast), 0.1 * math.log(f) + 1
    return inv, 1.0


def spans(st):
    """(sequence, first packed token, first row, end row)."""
    at = 0
    for b, (a, z) in enumerate(zip(st["s"].tolist(), st["e"].tolist())):
        yield b, at, a, z
        at += z - a


def plain_append(st):
    case, dt = st["case"], st["k"].dtype
    rot, D = case["rot"], case["D"]
    if st["positions"] is not None:
        at = st["positions"].double()
    else:
        at = torch.cat([torch.arange(a, z, device="cuda") for _, _, a, z in spans(st)]).double()
    inv, factor = frequencies(case)
    angle = at[:, None] * torch.from_numpy(inv).cuda()
    cos, sin = (angle.cos() * factor).float()[:, None], (angle.sin() * factor).float()[:, None]

    def rotate(x):
        x = x.float()
        if case["layout"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([r, x[..., rot:]], -1).to(dt)

    q, k = rotate(st["qn"]), rotate(st["kn"])
    for b, t, a, z in spans(st):
        n = z - a
        st["k"][0, b, :, :, a:z] = k[t:t + n].view(n, -1, D // 8, 8).permute(1, 2, 0, 3)
        st["v"][0, b, :, a:z] = st["vn"][t:t + n].transpose(0, 1)
    return {"q": q, "k": st["k"], "v": st["v"]}


def plain_compact(st):
    for b, t, a, z in spans(st):
        rows = st["keep"][t:t + z - a].long()
        st["k"][:, b, :, :, a:z] = st["k"][:, b].index_select(3, rows)
        st["v"][:, b, :, a:z] = st["v"][:, b].index_select(2, rows)
    return {"k": st["k"].view(torch.int16), "v": st["v"].view(torch.int16)}


def seen(st, t, a, z):
    """[new, z] truth values: which rows of the cache each new token attends."""
    n = z - a
    col = torch.arange(z, device="cuda")
    if st["bits"] is None:
        return col[None] <= torch.arange(a, z, device="cuda")[:, None]
    own_bits = st["bits"][t:t + n, None] >> (col - a).clamp(0, 63)[None] & 1
    return (col < a)[None] | (own_bits > 0)


def plain_attention(st):
    case = st["case"]
    H, G, D = case["H"], case["G"], case["D"]
    out = torch.empty_like(st["q"])
    for b, t, a, z in spans(st):
        n = z - a
        q = st["q"][t:t + n].float().view(n, H, G, D).permute(1, 2, 0, 3)
        hidden = ~seen(st, t, a, z)
        step = max(1, (1 << 29) // (G * n * z))  # heads at a time: 2 GiB of scores
        for h in range(0, H, step):
            k = st["k"][0, b, h:h + step, :, :z].float().permute(0, 2, 1, 3).reshape(-1, z, D)
            v = st["v"][0, b, h:h + step, :z].float()
            x = torch.matmul(q[h:h + step], k.transpose(1, 2)[:, None]) * st["scale"]
            x = x.masked_fill_(hidden, -math.inf)
            x = x.sub_(x.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(x, v[:, None]) / x.sum(-1, keepdim=True)
            out[t:t + n, h * G:(h + step) * G] = o.permute(2, 0, 1, 3).reshape(n, -1, D).to(out.dtype)
    return out


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "compact":
        return None  # copies
    st = prepare(case, seed)
    s, n, D, H, G = st["s"], st["e"] - st["s"], case["D"], case["H"], case["G"]
    first = np.concatenate([[0], np.cumsum(n)])
    if case["op"] == "append":
        inv, factor = frequencies(case)
        q, k = st["qn"].double(), st["kn"].double()
        K, V = st["k"].double(), st["v"].double()
        rows = np.concatenate([np.arange(a, a + m) for a, m in zip(s, n)])
        pos = st["positions"].double() if st["positions"] is not None else torch.from_numpy(rows).double().cuda()
        i = torch.arange(case["rot"] // 2, device="cuda")
        one, two = (i, i + case["rot"] // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        turn = torch.polar(torch.full((len(rows), len(inv)), factor, dtype=torch.float64, device="cuda"),
                           torch.outer(pos, torch.from_numpy(inv).cuda()))[:, None]
        for x in (q, k):
            w = torch.complex(x[..., one], x[..., two]) * turn
            x[..., one], x[..., two] = w.real, w.imag
        seq = torch.from_numpy(np.repeat(np.arange(len(s)), n)).cuda()
        at = torch.from_numpy(rows).cuda()
        K[0].permute(0, 3, 1, 2, 4)[seq, at] = k.view(len(rows), H, D // 8, 8)
        V[0].permute(0, 2, 1, 3)[seq, at] = st["vn"].double()
        return {"q": q, "k": K, "v": V}
    if work(case)["flops"] > 6e12:
        return None
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(len(s)):
        t, a, m, z = int(first[b]), int(s[b]), int(n[b]), int(s[b] + n[b])
        keys = st["k"][0, b, :, :, :z].double().transpose(1, 2).reshape(H, z, D)
        vals = st["v"][0, b, :, :z].double()
        for i in range(0, m, 256):
            j = min(m, i + 256)
            ok = torch.zeros(j - i, z, dtype=torch.bool, device="cuda")
            ok[:, :a] = True
            if st["bits"] is None:
                ok |= torch.ones(m, z, dtype=torch.bool, device="cuda").tril(a)[i:j]
            else:
                for c in range(m):
                    ok[:, a + c] = (st["bits"][t + i:t + j] >> c & 1).bool()
            for h in range(H):
                x = torch.einsum("ngd,kd->gnk", st["q"][t + i:t + j, h * G:(h + 1) * G].double(), keys[h]) * st["scale"]
                x = torch.where(ok, x, -math.inf)
                w = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
                out[t + i:t + j, h * G:(h + 1) * G] = torch.einsum("gnk,kd->ngd", w, vals[h])
    return out

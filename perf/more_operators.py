"""Measured cases of the operators that keep a cache within a bound: attention through a sliding window with a few first
rows that stay visible, attention that adds up the weight each cache row has received, and the eviction of the rows that
received least.

Cache layout of one layer, with 8 elements of 2 bytes per 16-byte chunk: K [B][H][D/8][S][8], V [B][H][S][D]; the rows'
accumulated weight: float32 [B][H][S] a layer.
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
    return [
        # one decode token over a narrow window of short sequences: latency
        dict(name="window_decode_short", op="window", **gpt2, ctx=100, ctx_hi=1000, new=1, new_hi=1, window=200, sinks=4,
             ranges=1),
        # one decode token of a full batch, many heads; contexts below and above the window
        dict(name="window_decode_batch", op="window", **bloom, ctx=64, ctx_hi=1791, new=1, new_hi=1, window=512, sinks=4,
             ranges=2),
        # ragged prompts, some shorter than the window, which ends inside tiles
        dict(name="window_prompts", op="window", **opt, ctx=0, ctx_hi=0, new=16, new_hi=2048, window=500, sinks=1,
             ranges=3),
        # a chunk of a long prompt far behind its first rows, grouped heads
        dict(name="window_chunk_far", op="window", **grouped, B=1, S=131072, ctx=120000, ctx_hi=120000, new=4096,
             new_hi=4096, window=4096, sinks=16, ranges=4),
        # one decode token over short contexts, its weights added up: latency
        dict(name="scored_decode_short", op="scored", **gpt2, ctx=100, ctx_hi=1000, new=1, new_hi=1, last=0, ranges=5),
        # one decode token of a full batch, many heads
        dict(name="scored_decode_batch", op="scored", **bloom, ctx=64, ctx_hi=1791, new=1, new_hi=1, last=0, ranges=6),
        # one decode token over long contexts, grouped heads
        dict(name="scored_decode_long", op="scored", **grouped, B=2, S=131072, ctx=100000, ctx_hi=131000, new=1, new_hi=1,
             last=0, ranges=7),
        # ragged prompts, every token's weights added up
        dict(name="scored_prompts", op="scored", **bloom, ctx=0, ctx_hi=0, new=64, new_hi=1536, last=0, ranges=8),
        # the last chunk of a long prompt, whose last 64 tokens alone are counted
        dict(name="scored_chunk_last", op="scored", **grouped, B=1, S=32768, ctx=28672, ctx_hi=28672, new=4096,
             new_hi=4096, last=64, ranges=9),
        # small caches brought back to their bound after some decode steps
        dict(name="evict_steps", op="evict", **gpt2, L=1, rows=401, rows_hi=433, keep=400, keep_hi=400, sinks=4,
             recent=100, ranges=10),
        # ragged prompts' rows halved in every layer of a block
        dict(name="evict_prompts", op="evict", **opt, L=8, rows=520, rows_hi=2040, keep=257, keep_hi=1020, sinks=4,
             recent=128, ranges=11),
        # long contexts cut to a small part, few heads
        dict(name="evict_long", op="evict", **grouped, B=2, S=131072, L=4, rows=100000, rows_hi=131000, keep=8192,
             keep_hi=16384, sinks=16, recent=1024, ranges=12),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["window", "scored", "evict"])
    G, D = rng.choice([1, 1, 2, 4, 5, 8]), rng.choice([64, 128, 64, 128, 80, 96])
    case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), B=spread(1, 32), H=spread(1, 40), G=G, D=D,
                ranges=rng.randrange(1 << 30))
    if op == "evict":
        n, L = spread(2, 60000), spread(1, 8)
        while L * case["B"] * case["H"] * D * n > 1 << 28:
            L, case["B"], n = max(1, L // 2), max(1, case["B"] // 2), max(2, n // 2)
        keep = max(1, int(n * rng.choice([0.1, 0.25, 0.5, 0.9])))
        sinks = min(rng.choice([0, 1, 4, 16]), keep // 4)
        case |= dict(L=L, rows=max(keep, n // rng.choice([1, 2])), rows_hi=n, keep=max(1, keep // rng.choice([1, 2])),
                     keep_hi=keep, sinks=sinks, S=n + rng.randrange(0, 70))
        case["recent"] = min(rng.choice([0, 8, 64, 512]), case["keep"] - min(sinks, case["keep"]))
        case["sinks"] = min(sinks, case["keep"])
        return case
    top = 1 if rng.random() < 0.4 else spread(1, 8192)
    while case["B"] * case["H"] * G * top * top > 64 * 2048 * 4096:
        case["B"] = max(1, case["B"] // 2)
        top = max(1, top // 2) if case["B"] == 1 else top
    ctx = rng.choice([0, spread(1, 32768), spread(1, 32768)])
    while ctx and (case["B"] * case["H"] * G * top * (top + ctx) > 64 * 2048 * 8192
                   or case["B"] * case["H"] * D * (top + ctx) > 1 << 28):
        ctx //= 2
    case |= dict(ctx=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx, new=max(1, top // rng.choice([1, 2, 8])), new_hi=top,
                 S=ctx + top + rng.randrange(0, 70))
    if op == "window":
        case |= dict(window=spread(1, 8192), sinks=rng.choice([0, 1, 4, 16, 130]))
    else:
        case |= dict(last=rng.choice([0, 0, 1, 32, 64]))
    return case


def lengths(case):
    """Rows before the new ones and new rows of each sequence (evict: rows in use, rows kept), int32 arrays."""
    r = random.Random(case["ranges"])
    one, two = (("rows", "keep") if case["op"] == "evict" else ("ctx", "new"))
    a = [r.randint(case[one], case[one + "_hi"]) for _ in range(case["B"])]
    b = [r.randint(case[two], case[two + "_hi"]) for _ in range(case["B"])]
    if case["op"] == "evict":
        b = [min(x, y) for x, y in zip(a, b)]
    return np.array(a, np.int32), np.array(b, np.int32)


def work(case):
    s, n = (x.astype(np.int64) for x in lengths(case))
    H, D, Hq = case["H"], case["D"], case["H"] * case["G"]
    if case["op"] == "evict":
        # kept K and V rows read and written (those of the first rows stay where they are), the weights read, the kept
        # ones and the zeros behind them written, the list
        moved = int((np.where(n < s, n - case["sinks"], 0)).sum())
        per = case["L"] * H
        return {"bytes": per * (2 * 2 * 2 * D * moved + 8 * int(s.sum()) + 4 * int(n.sum())), "flops": 0}
    T = int(n.sum())
    if case["op"] == "scored":
        pairs = int((s * n + n * (n + 1) // 2).sum())
        rows = int((s + n).sum())
        counted = np.minimum(n, case["last"]) if case["last"] else n
        # every weight once for the output and once, as a sum over the counted tokens, for its row
        sums = int((counted * (s + n) - counted * (counted - 1) // 2).sum())
        return {"bytes": 2 * (2 * T * Hq * D + 2 * rows * H * D) + 8 * H * rows, "flops": Hq * (4 * D * pairs + sums)}
    pairs = rows = 0
    w, sinks = case["window"], case["sinks"]
    for a, m in zip(s.tolist(), n.tolist()):
        r = np.arange(a, a + m)
        first = np.maximum(0, r - w + 1)
        pairs += int((r + 1 - first + np.minimum(first, sinks)).sum())
        rows += a + m - int(first[0]) + min(int(first[0]), sinks)
    return {"bytes": 2 * (2 * T * Hq * D + 2 * rows * H * D), "flops": 4 * D * Hq * pairs}


# ---- inputs -------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, B, H, D, S = DTYPES[case["dtype"]], case["B"], case["H"], case["D"], case["S"]
    Hq, L = H * case["G"], case.get("L", 1)
    a, n = lengths(case)

    def normal(*shape):
        return torch.empty(*shape, dtype=dt, device="cuda").normal_(generator=g)

    st = dict(case=case, k=normal(L, B, H, D // 8, S, 8), v=normal(L, B, H, S, D))
    if case["op"] == "evict":
        # weights as attention leaves them: few rows with much, most with little, and some alike or without any
        x = torch.rand(L, B, H, S, generator=g, device="cuda")
        few = torch.rand(L, B, H, S, generator=g, device="cuda")
        x = torch.where(few < 0.1, (x * 8).floor() / 8, x ** 8 * 30)
        st |= dict(rows=a, kept=n, mass=x, mass_out=torch.empty_like(x).fill_(0.0),
                   keep=torch.empty(L, H, int(n.sum()), dtype=torch.int32, device="cuda"))
    else:
        T = int(n.sum())
        st |= dict(s=a, e=a + n, q=normal(T, Hq, D) * 2, out=torch.empty(T, Hq, D, dtype=dt, device="cuda"),
                   scale=D ** -0.5)
        if case["op"] == "scored":
            # what earlier tokens left; a prompt is the first
            st["mass"] = torch.rand(B, H, S, generator=g, device="cuda") * float(case["ctx"] > 0)
    if own:  # what a program keeps between its calls: the cache's description, the workspace
        import kv_cache_streaming_gb300 as dv
        st["cache"] = dv.Cache(L, B, H, D, S, 2, st["k"], st["v"])
        if case["op"] != "evict":
            size = dv.dv_scored_attention_workspace if case["op"] == "scored" else dv.dv_attention_workspace
            st["workspace"] = torch.empty(size(st["cache"], a, a + n, Hq), dtype=torch.uint8, device="cuda")
    return st


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(st):
    case = st["case"]
    if case["op"] == "evict":
        if own:
            import kv_cache_streaming_gb300 as dv
            dv.dv_kv_evict(st["cache"], 0, case["L"], st["rows"], st["kept"], case["sinks"], case["recent"], st["mass"],
                           st["keep"], mass_out=st["mass_out"])
        else:
            plain_evict(st)
        return {"keep": st["keep"], "mass": st["mass_out"], "k": st["k"].view(torch.int16),
                "v": st["v"].view(torch.int16)}
    if not own:
        plain_attention(st)
    else:
        import kv_cache_streaming_gb300 as dv
        if case["op"] == "window":
            dv.dv_window_attention(st["cache"], 0, st["s"], st["e"], st["q"], st["out"], st["scale"], case["window"],
                                   case["sinks"], st["workspace"])
        else:
            dv.dv_scored_attention(st["cache"], 0, st["s"], st["e"], st["q"], st["out"], st["scale"], st["mass"],
                                   st["workspace"], last=case["last"])
    return {"out": st["out"], "mass": st["mass"]} if case["op"] == "scored" else st["out"]


def spans(st):
    """(sequence, first packed token, first new row, end row)."""
    at = 0
    for b, (a, z) in enumerate(zip(st["s"].tolist(), st["e"].tolist())):
        yield b, at, a, z
        at += z - a


def plain_attention(st):
    """A block of tokens at a time over the rows that any of them attends."""
    case = st["case"]
    H, G, D = case["H"], case["G"], case["D"]
    w, sinks = (case["window"], case["sinks"]) if case["op"] == "window" else (1 << 30, 0)
    for b, t, a, z in spans(st):
        block = min(z - a, max(256, w // 2) if w < z else z - a)
        for i in range(a, z, block):
            j = min(z, i + block)
            n, lo = j - i, max(0, i - w + 1)
            col = torch.arange(lo, j, device="cuda")
            if lo > 0 and sinks:
                col = torch.cat([torch.arange(min(sinks, lo), device="cuda"), col])
            row = torch.arange(i, j, device="cuda")[:, None]
            hidden = (col > row) | ((col <= row - w) & (col >= sinks))
            tok = slice(t + i - a, t + j - a)
            q = st["q"][tok].float().view(n, H, G, D).permute(1, 2, 0, 3)
            step = max(1, (1 << 29) // (G * n * len(col)))  # heads at a time: 2 GiB of scores
            for h in range(0, H, step):
                heads = slice(h, h + step)
                if len(col) == j:  # every row so far
                    k, v = st["k"][0, b, heads, :, :j], st["v"][0, b, heads, :j]
                else:
                    k, v = st["k"][0, b, heads].index_select(2, col), st["v"][0, b, heads].index_select(1, col)
                k = k.float().permute(0, 2, 1, 3).reshape(-1, len(col), D)
                x = torch.matmul(q[heads], k.transpose(1, 2)[:, None]) * st["scale"]
                x = x.masked_fill_(hidden, -math.inf)
                x = x.sub_(x.amax(-1, keepdim=True)).exp_()
                total = x.sum(-1, keepdim=True)
                o = torch.matmul(x, v.float()[:, None]) / total
                st["out"][tok, h * G:(h + step) * G] = o.permute(2, 0, 1, 3).reshape(n, -1, D).to(st["out"].dtype)
                if case["op"] == "scored":
                    last = min(n, case["last"]) if case["last"] else n
                    st["mass"][b, heads, :j] += (x[:, :, n - last:] / total[:, :, n - last:]).sum((1, 2))


def plain_evict(st):
    case, at = st["case"], 0
    sinks, recent = case["sinks"], case["recent"]
    for b, (n, m) in enumerate(zip(st["rows"].tolist(), st["kept"].tolist())):
        x = st["mass"][:, b, :, :n]
        if m < n:
            top = x[..., sinks:n - recent].sort(dim=-1, descending=True, stable=True).indices[..., :m - sinks - recent]
            rows = torch.arange(n, device="cuda").expand(x.shape)
            rows = torch.cat([rows[..., :sinks], top.sort(dim=-1).values + sinks, rows[..., n - recent:]], -1)
            st["k"][:, b, :, :, :m] = st["k"][:, b].gather(3, rows[:, :, None, :, None].expand(
                -1, -1, case["D"] // 8, -1, 8))
            st["v"][:, b, :, :m] = st["v"][:, b].gather(2, rows[..., None].expand(-1, -1, -1, case["D"]))
        else:
            rows = torch.arange(n, device="cuda").expand(x.shape)
        st["keep"][:, :, at:at + m] = rows
        st["mass_out"][:, b, :, :m] = x.gather(-1, rows)
        st["mass_out"][:, b, :, m:n] = 0.0
        at += m


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "evict":
        return None  # copies and whole numbers
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    s, n, D, H, G = st["s"], st["e"] - st["s"], case["D"], case["H"], case["G"]
    first = np.concatenate([[0], np.cumsum(n)])
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    mass = st["mass"].double() if case["op"] == "scored" else None
    for b in range(len(s)):
        t, a, m, z = int(first[b]), int(s[b]), int(n[b]), int(s[b] + n[b])
        for i in range(0, m, 256):
            j = min(m, i + 256)
            r = torch.arange(a + i, a + j, device="cuda")
            rows = torch.arange(z, device="cuda")
            ok = rows <= r[:, None]
            if case["op"] == "window":
                ok &= (r[:, None] - rows < case["window"]) | (rows < case["sinks"])
            rows = rows[ok.any(0)]
            ok = ok[:, rows]
            counted = torch.arange(i, j, device="cuda") >= (m - case["last"] if case.get("last") else 0)
            for h in range(H):
                keys = st["k"][0, b, h].double().index_select(1, rows)
                vals = st["v"][0, b, h].double().index_select(0, rows)
                x = torch.einsum("ngce,cke->gnk", st["q"][t + i:t + j, h * G:(h + 1) * G].double().unflatten(
                    -1, (D // 8, 8)), keys) * st["scale"]
                x = torch.where(ok, x, -math.inf)
                w = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
                out[t + i:t + j, h * G:(h + 1) * G] = torch.einsum("gnk,kd->ngd", w, vals)
                if mass is not None:
                    mass[b, h].index_add_(0, rows, torch.einsum("gnk,n->k", w, counted.double()))
    return out if mass is None else {"out": out, "mass": mass}

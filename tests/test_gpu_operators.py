"""The operators over the cache against plain 64-bit forms (tests/operator_refs.py,
which derives the bounds): types, head layouts, odd sizes, strides, empty rows and
ranges, values that a mask hides, streams, graphs, and what is refused."""
import math

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv
from tests import operator_refs as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    dv.dv_attention_check()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ws(cache, s, e, q_heads):
    """The workspace, filled with NaN bits: it needs no initial value."""
    n = dv.dv_attention_workspace(cache, s, e, q_heads)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None


def _draw(rng, lo, hi, B, some_empty=False):
    v = rng.integers(lo, hi + 1, size=B).astype(np.int32)
    if some_empty and B > 1:
        v[rng.integers(0, B)] = 0
    return v


def _attend(cache, layer, s, e, q, scale, tree=None, prompt=False, out=None):
    out = torch.full_like(q, math.nan) if out is None else out
    ws = _ws(cache, s, e, q.shape[1])
    if prompt:
        dv.dv_prompt_attention(cache, layer, s, e, q, out, scale, ws)
    else:
        dv.dv_tree_attention(cache, layer, s, e, q, out, scale, ws, tree=tree)
    return out


# ---- append ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B, H, G, D, S, ctx, new, rot, inter, scaling, far", [
    (2, 3, 1, 64, 40, (0, 20), (1, 1), 64, False, "none", False),
    (3, 5, 2, 64, 70, (0, 33), (1, 37), 32, True, "linear", False),
    (1, 1, 1, 8, 9, (0, 0), (9, 9), 8, False, "none", False),
    (4, 2, 4, 128, 130, (0, 60), (5, 64), 128, False, "parts", True),
    (2, 2, 3, 80, 300, (3, 90), (100, 200), 20, False, "ntk", False),  # pairs across chunks
    (2, 2, 1, 96, 50, (1, 9), (2, 40), 44, True, "none", True),        # a chunk half rotated
    (40, 2, 2, 64, 33, (0, 8), (0, 25), 64, False, "none", False),     # more than 32 sequences
    (2, 1, 1, 320, 20, (0, 3), (1, 17), 256, True, "none", False),     # long heads
    (1, 71, 1, 64, 12, (2, 2), (3, 3), 64, False, "none", True),
])
def test_append(dtype, B, H, G, D, S, ctx, new, rot, inter, scaling, far):
    rng = np.random.default_rng(B * 1000 + D)
    gen = _gen(D + B)
    s = _draw(rng, *ctx, B)
    e = s + np.minimum(_draw(rng, *new, B, some_empty=True), S - s).astype(np.int32)
    T, Hq = int((e - s).sum()), H * G
    cache, K, V = R.make_cache(dtype, 2, B, H, D, S, gen, stride=B * H * D * S + 64)
    qkv = torch.empty(T, (Hq + 2 * H) * D + 8, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + H) * D].view(T, H, D)
    v = qkv[:, (Hq + H) * D:(Hq + 2 * H) * D].view(T, H, D)
    if rot < D:  # what is not rotated keeps its bits, and touches nothing else
        q[:, :, rot:] = math.inf
        k[:, 0, rot:] = math.nan
    pos = torch.from_numpy(np.concatenate([np.arange(a, z) for a, z in zip(s, e)]).astype(np.int32)).cuda()
    if far:
        pos = torch.randint(-5, 1 << 20, (T,), generator=gen, device="cuda", dtype=torch.int32)
    K0, V0 = K.clone(), V.clone()
    rope = dv.Rope(rot, interleaved=inter, base=10000.0, scaling=scaling, factor=4.0, original_max=2048)
    q_out = dv.dv_kv_append(cache, 1, s, e, k, v, q=q, rope=rope, positions=pos if far else None)
    f, m = R.rope_freqs(rot, 10000.0, scaling, 4.0, 2048)
    for x, got in ((q, q_out), (k, None)):
        want, tol = R.rotate_ref(x, pos, rot, inter, f, m)
        if got is None:
            got = torch.cat([K[1, b, :, :, a:z].permute(2, 0, 1, 3).reshape(z - a, H, D)
                             for b, _, a, z in R.spans(s, e)])
        R.assert_within(got[..., :rot], want[..., :rot], tol[..., :rot], "rotated")
        assert torch.equal(got[..., rot:].view(torch.int16), x[..., rot:].view(torch.int16))
    for b, t, a, z in R.spans(s, e):
        assert torch.equal(V[1, b, :, a:z], v[t:t + z - a].transpose(0, 1))
        for now, was in ((K, K0), (V, V0)):
            dim = 3 if now is K else 2
            for lo, hi in ((0, a), (z, S)):
                assert torch.equal(now.select(0, 1)[b].narrow(dim - 1, lo, hi - lo),
                                   was.select(0, 1)[b].narrow(dim - 1, lo, hi - lo))
    assert torch.equal(K[0], K0[0]) and torch.equal(V[0], V0[0])


@pytest.mark.parametrize("seed", range(12))
def test_random_append(seed):
    rng = np.random.default_rng(seed)
    gen = _gen(seed)
    dtype = ["fp16", "bf16"][rng.integers(2)]
    B, H, G, D = int(rng.integers(1, 9)), int(rng.integers(1, 9)), int(rng.integers(1, 6)), 8 * int(rng.integers(1, 25))
    rot = 2 * int(rng.integers(1, min(D, 256) // 2 + 1))
    inter, scaling = bool(rng.integers(2)), str(rng.choice(["none", "linear", "parts"]))
    s = rng.integers(0, 50, size=B).astype(np.int32)
    e = s + rng.integers(0, int(rng.choice([2, 5, 60])), size=B).astype(np.int32)
    S, T = int(e.max()) + int(rng.integers(0, 9)) + 1, int((e - s).sum())
    cache, K, V = R.make_cache(dtype, 1, B, H, D, S, gen)
    q = torch.empty(T, H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    k, v = (torch.empty(T, H, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) for _ in range(2))
    pos = torch.randint(0, 1 << 19, (T,), generator=gen, device="cuda", dtype=torch.int32)
    q_out = dv.dv_kv_append(cache, 0, s, e, k, v, q=q, positions=pos,
                            rope=dv.Rope(rot, interleaved=inter, scaling=scaling, factor=8.0, original_max=4096))
    f, m = R.rope_freqs(rot, 10000.0, scaling, 8.0, 4096)
    want, tol = R.rotate_ref(q, pos, rot, inter, f, m)
    R.assert_within(q_out[..., :rot], want[..., :rot], tol[..., :rot])
    assert torch.equal(q_out[..., rot:], q[..., rot:])
    want, tol = R.rotate_ref(k, pos, rot, inter, f, m)
    for b, t, a, z in R.spans(s, e):
        got = K[0, b, :, :, a:z].permute(2, 0, 1, 3).reshape(z - a, H, D)
        R.assert_within(got, want[t:t + z - a], tol[t:t + z - a] + (torch.arange(D, device="cuda") >= rot) * 0.0)
        assert torch.equal(V[0, b, :, a:z].transpose(0, 1), v[t:t + z - a])


def test_append_without_rotation_or_queries_copies():
    gen = _gen(3)
    s, e = np.array([5, 0], np.int32), np.array([25, 11], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 2, 3, 64, 30, gen)
    k, v = (torch.empty(31, 3, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    assert dv.dv_kv_append(cache, 0, s, e, k, v) is None
    q = torch.empty(31, 6, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    assert torch.equal(dv.dv_kv_append(cache, 0, s, e, k, v, q=q), q)
    for b, t, a, z in R.spans(s, e):
        assert torch.equal(K[0, b, :, :, a:z].permute(2, 0, 1, 3).reshape(z - a, 3, 64), k[t:t + z - a])
        assert torch.equal(V[0, b, :, a:z].transpose(0, 1), v[t:t + z - a])


# ---- attention -------------------------------------------------------------------------

PROMPTS = [
    # B, H, G, D, S, ctx, new
    (1, 1, 1, 64, 1, (0, 0), (1, 1)),
    (2, 2, 1, 64, 150, (0, 0), (127, 130)),
    (3, 3, 1, 128, 300, (0, 0), (1, 300)),
    (2, 2, 4, 128, 700, (0, 200), (100, 500)),
    (3, 2, 3, 64, 421, (0, 100), (0, 321)),
    (2, 1, 71, 64, 90, (0, 30), (1, 60)),
    (1, 1, 128, 128, 40, (0, 0), (33, 33)),
    (2, 2, 2, 8, 140, (0, 4), (1, 136)),
    (2, 2, 1, 72, 517, (0, 129), (250, 388)),
    (2, 1, 5, 96, 260, (5, 5), (200, 255)),
    (2, 1, 2, 120, 513, (256, 257), (255, 256)),
    (36, 2, 1, 64, 70, (0, 10), (0, 60)),
    (1, 2, 1, 128, 2048, (0, 0), (2048, 2048)),
    (1, 1, 2, 64, 5000, (4500, 4500), (300, 300)),
    # more units than the GPU has SMs, some of one row tile with many K/V tiles
    (4, 64, 1, 128, 1500, (600, 900), (40, 600)),
    (6, 50, 1, 64, 1300, (0, 900), (1, 390)),
    (3, 60, 3, 128, 700, (0, 500), (20, 90)),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B, H, G, D, S, ctx, new", PROMPTS)
def test_prompt_attention(dtype, B, H, G, D, S, ctx, new):
    rng = np.random.default_rng(S)
    gen = _gen(S + D)
    s = _draw(rng, *ctx, B)
    e = s + np.minimum(_draw(rng, *new, B, some_empty=new[0] == 0), S - s).astype(np.int32)
    cache, K, V = R.make_cache(dtype, 2, B, H, D, S, gen)
    q = torch.empty(int((e - s).sum()), H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) * 2
    scale = D ** -0.5
    want, tol = R.attention_ref(K[1], V[1], s, e, q, scale)
    for b, _, a, z in R.spans(s, e):  # nothing past a sequence's rows is attended
        K[:, b, :, :, z:] = math.nan
        V[:, b, :, z:] = math.nan
    got = _attend(cache, 1, s, e, q, scale, prompt=True)
    R.assert_within(got, want, tol)
    assert torch.equal(_attend(cache, 1, s, e, q, scale, prompt=True), got)  # the same bits again


TREES = [
    # B, H, G, D, S, ctx, new
    (2, 3, 1, 64, 50, (0, 40), (1, 1)),
    (4, 2, 1, 128, 400, (0, 390), (1, 9)),
    (3, 2, 4, 128, 1000, (100, 936), (1, 64)),
    (2, 2, 8, 64, 333, (0, 269), (33, 64)),
    (2, 1, 71, 64, 300, (0, 200), (1, 3)),
    (1, 1, 128, 128, 200, (100, 130), (64, 64)),
    (2, 2, 3, 40, 260, (120, 129), (1, 17)),
    (2, 2, 1, 88, 260, (64, 200), (5, 60)),
    (40, 1, 2, 64, 100, (0, 90), (0, 10)),
    (1, 1, 1, 128, 20000, (19900, 19900), (1, 1)),
    (1, 2, 4, 128, 9000, (8900, 8900), (31, 31)),
    (5, 70, 1, 128, 1200, (0, 1130), (1, 20)),   # more units than the GPU has SMs
    (4, 64, 2, 64, 900, (0, 830), (0, 64)),
    (3, 60, 4, 128, 800, (300, 730), (20, 64)),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("masked", [True, False], ids=["tree", "chain"])
@pytest.mark.parametrize("B, H, G, D, S, ctx, new", TREES)
def test_tree_attention(dtype, masked, B, H, G, D, S, ctx, new):
    rng = np.random.default_rng(S + B)
    gen = _gen(S + D)
    s = _draw(rng, *ctx, B)
    e = s + np.minimum(_draw(rng, *new, B, some_empty=new[0] == 0), S - s).astype(np.int32)
    cache, K, V = R.make_cache(dtype, 1, B, H, D, S, gen)
    q = torch.empty(int((e - s).sum()), H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) * 2
    bits = sum((R.random_tree(int(z - a), rng)[0] for a, z in zip(s, e)), []) if masked else None
    want, tol = R.attention_ref(K[0], V[0], s, e, q, D ** -0.5, bits)
    for b, _, a, z in R.spans(s, e):
        K[:, b, :, :, z:] = math.inf
        V[:, b, :, z:] = math.nan
    if masked:  # bits past the sequence's tokens count for nothing
        n = np.repeat(e - s, e - s).tolist()
        bits = [x | (((1 << 64) - 1) ^ ((1 << m) - 1)) for x, m in zip(bits, n)]
    tree = R.bits_tensor(bits) if masked else None
    got = _attend(cache, 0, s, e, q, D ** -0.5, tree=tree)
    R.assert_within(got, want, tol)
    assert torch.equal(_attend(cache, 0, s, e, q, D ** -0.5, tree=tree), got)


@pytest.mark.parametrize("dtype, G, D", [("fp16", 1, 64), ("bf16", 4, 128), ("fp16", 16, 96)])
@pytest.mark.parametrize("ctx", [0, 1, 100, 128, 250])
def test_hidden_values_have_no_effect(dtype, G, D, ctx):
    """NaN and infinities in tree rows reach exactly the tokens that attend
    them; tokens that attend nothing have zeros."""
    B, H, n, S = 2, 2, 40, 300
    gen = _gen(ctx + D)
    rng = np.random.default_rng(ctx)
    s = np.array([ctx, ctx + 3], np.int32)
    e = s + n
    cache, K, V = R.make_cache(dtype, 1, B, H, D, S, gen)
    q = torch.empty(2 * n, H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    bits = R.random_tree(n, rng)[0] + R.random_tree(n, rng)[0]
    bits[3] = 0       # with an empty context: attends no row
    bits[n + 2] = 1 << 1
    V[0, 0, :, ctx + 17, 5] = math.nan
    V[0, 0, 1, ctx + 20, 0] = math.inf
    V[0, 1, 0, ctx + 3 + 30, D - 1] = -math.inf
    K[0, 0, 1, :, ctx + 25] = math.nan
    K[0, 1, 0, :, ctx + 3 + 11] = math.inf
    want, tol = R.attention_ref(K[0], V[0], s, e, q, D ** -0.5, bits)
    got = _attend(cache, 0, s, e, q, D ** -0.5, tree=R.bits_tensor(bits))
    if ctx == 0:
        assert not got[3].any()
    R.assert_within(got, want, tol)


@pytest.mark.parametrize("ctx, n", [(0, 300), (130, 200), (5, 1)])
def test_later_prompt_rows_have_no_effect(ctx, n):
    """In a prompt too: a NaN value or key reaches its own and later tokens only."""
    H, D, S = 2, 128, ctx + n + 9
    gen = _gen(n)
    s, e = np.array([ctx], np.int32), np.array([ctx + n], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 1, H, D, S, gen)
    at = ctx + (2 * n) // 3
    V[0, 0, 0, at, 3] = math.nan
    V[0, 0, 1, at, 4] = math.inf
    q = torch.empty(n, 2 * H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    want, tol = R.attention_ref(K[0], V[0], s, e, q, D ** -0.5)
    got = _attend(cache, 0, s, e, q, D ** -0.5, prompt=True)
    R.assert_within(got, want, tol)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_growing_and_falling_scores(dtype):
    """Scores that rise along the rows (the running maximum moves at every
    step), that fall, and that are far apart."""
    H, D, S, n = 3, 64, 1024, 40
    gen = _gen(9)
    cache, K, V = R.make_cache(dtype, 1, 1, H, D, S, gen)
    ramp = torch.linspace(0.0, 12.0, S, device="cuda", dtype=torch.float64)
    for h, f in enumerate((ramp, ramp.flip(0), (ramp * 7) % 5 - 2)):
        k = K[0, 0, h].double()
        k[0, :, 0] = f
        K[0, 0, h] = k.to(K.dtype)
    s, e = np.array([S - n], np.int32), np.array([S], np.int32)
    q = torch.empty(n, H, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    q[:, :, 0] = 40.0
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 0.125)
    R.assert_within(_attend(cache, 0, s, e, q, 0.125), want, tol)
    R.assert_within(_attend(cache, 0, s, e, q, 0.125, prompt=True), want, tol)


@pytest.mark.parametrize("seed", range(32))
def test_random_attention(seed):
    """Seeded draws over types, head sizes and groups, lengths, masks, layers
    with a gap between them, and strided queries."""
    rng = np.random.default_rng(1000 + seed)
    gen = _gen(seed)
    dtype = ["fp16", "bf16"][rng.integers(2)]
    B, H, G = int(rng.integers(1, 7)), int(rng.integers(1, 7)), int(rng.choice([1, 2, 3, 4, 7, 8, 16]))
    D = 8 * int(rng.integers(1, 17))
    prompt = bool(rng.integers(2))
    most = int(rng.integers(1, 500)) if prompt else int(rng.integers(1, 65))
    ctx = int(rng.choice([0, int(rng.integers(1, 700))]))
    s = rng.integers(0, ctx + 1, size=B).astype(np.int32)
    e = s + rng.integers(0 if B > 1 else 1, most + 1, size=B).astype(np.int32)
    if e.sum() == s.sum():
        e[0] += 1
    S, T = int(e.max()) + int(rng.integers(0, 40)), int((e - s).sum())
    cache, K, V = R.make_cache(dtype, 3, B, H, D, S, gen, stride=B * H * D * S + 8 * int(rng.integers(0, 5)))
    wide = torch.empty(T, (H * G + 3) * D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    q = wide[:, D:(H * G + 1) * D].view(T, H * G, D)
    masked = not prompt and bool(rng.integers(2))
    bits = sum((R.random_tree(int(z - a), rng)[0] for a, z in zip(s, e)), []) if masked else None
    layer, scale = int(rng.integers(3)), float(rng.uniform(0.3, 2.0)) * D ** -0.5
    want, tol = R.attention_ref(K[layer], V[layer], s, e, q, scale, bits)
    for b, _, a, z in R.spans(s, e):
        K[:, b, :, :, z:], V[:, b, :, z:] = math.nan, math.nan
    out = torch.empty(T, H * G, D, dtype=R.DT[dtype], device="cuda")
    _attend(cache, layer, s, e, q, scale, tree=R.bits_tensor(bits) if masked else None, prompt=prompt, out=out)
    R.assert_within(out, want, tol)


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own, in flight together."""
    gen = _gen(77)
    jobs = []
    for i, (H, D, ctx, n) in enumerate([(8, 128, 3000, 5), (20, 64, 900, 33)]):
        s, e = np.array([ctx, 7], np.int32), np.array([ctx + n, 8 + n], np.int32)
        cache, K, V = R.make_cache("bf16", 1, 2, H, D, ctx + n, gen)
        q = torch.empty(2 * n + 1, H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        want, tol = R.attention_ref(K[0], V[0], s, e, q, D ** -0.5)
        jobs.append((cache, s, e, q, D ** -0.5, want, tol, torch.empty_like(q), _ws(cache, s, e, H), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for r in range(20):
        for cache, s, e, q, scale, _, _, out, ws, stream in jobs:
            dv.dv_tree_attention(cache, 0, s, e, q, out, scale, ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, _, _, _, want, tol, out, _, _ in jobs:
        R.assert_within(out, want, tol)


def test_strided_queries_and_output_leave_the_rest():
    gen = _gen(12)
    s, e = np.array([300, 0, 7], np.int32), np.array([320, 31, 8], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 3, 2, 64, 400, gen)
    T = 52
    wide = torch.empty(T, 5 * 64 + 24, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    q = wide[:, 64:5 * 64].view(T, 4, 64)
    buf = torch.full((T + 2, 7 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:T + 1, 64:5 * 64].view(T, 4, 64)
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 0.125)
    for prompt in (False, True):
        out.fill_(math.nan)
        _attend(cache, 0, s, e, q, 0.125, prompt=prompt, out=out)
        R.assert_within(out, want, tol)
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()
        assert (buf[:, :64] == 7).all() and (buf[:, 5 * 64:] == 7).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: the last head's rows, far along."""
    H, D, S = 9, 128, 1 << 21
    gen = _gen(5)
    k = torch.zeros(H * D * S, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(H * D * S, dtype=torch.bfloat16, device="cuda")
    cache = dv.Cache(1, 1, H, D, S, 2, k, v)
    K, V = k.view(1, 1, H, D // 8, S, 8), v.view(1, 1, H, S, D)
    n, at = 6, S - 6
    s, e = np.array([at], np.int32), np.array([S], np.int32)
    new = torch.empty(n, 3 * H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    V[0, 0, :, :at] = 1.0
    q = dv.dv_kv_append(cache, 0, s, e, new[:, H:2 * H], new[:, 2 * H:], q=new[:, :H], rope=dv.Rope(128))
    # the context's keys are zero (score 0), its values one; the new keys weigh about as much
    q, scale = (q * 3).contiguous(), 0.4
    got = _attend(cache, 0, s, e, q, scale)
    ok = torch.tril(torch.ones(n, n, dtype=torch.bool, device="cuda"))
    kk = K[0, 0, :, :, at:].double().permute(0, 2, 1, 3).reshape(H, n, D)
    x = (torch.einsum("nhd,hkd->hnk", q.double(), kk) * scale).masked_fill(~ok, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=0)
    w, w0 = torch.exp(x - m), at * torch.exp(-m)
    o = ((torch.einsum("hnk,hkd->hnd", w, V[0, 0, :, at:].double()) + w0) /
         (w.sum(-1, keepdim=True) + w0)).transpose(0, 1)
    # as attention_ref (|v| at most va), but for the 32-bit sums: of 2^21 like terms, added in
    # blocks of 32 or more, 2^16 additions to the weights' sum and as many to the output's
    va = max(1.0, float(V[0, 0, :, at:].double().abs().amax()))
    qk = float(torch.einsum("nhd,hkd->hnk", q.double().abs(), kk.abs()).amax())
    tol = torch.full_like(o, va * (2 * 2.0 ** -8 + 2 * 128 * 2.0 ** -24 * qk * scale + 2 * 2.0 ** -8))
    R.assert_within(got, o, tol)
    keep = torch.tensor([S - 6, S - 3, S - 1], dtype=torch.int32, device="cuda")
    rows = (K[0, 0, :, :, S - 3].clone(), V[0, 0, :, S - 1].clone())
    dv.dv_kv_compact(cache, 0, 1, s, s + 3, keep)
    assert torch.equal(K[0, 0, :, :, at + 1], rows[0]) and torch.equal(V[0, 0, :, at + 2], rows[1])
    del k, v, K, V, cache
    torch.cuda.empty_cache()


def test_side_stream_and_graph():
    """Work goes to the given stream, in order with it; a captured pass replays
    on new values in the same buffers."""
    gen = _gen(21)
    B, H, D, S = 2, 4, 64, 600
    s, e = np.array([500, 33], np.int32), np.array([517, 40], np.int32)
    T = 24
    cache, K, V = R.make_cache("fp16", 1, B, H, D, S, gen)
    qkv = torch.empty(T, 3 * H, D, dtype=torch.float16, device="cuda").normal_(generator=gen)
    q, out = torch.empty(T, H, D, dtype=torch.float16, device="cuda"), torch.empty(T, H, D, dtype=torch.float16, device="cuda")
    rope, keep = dv.Rope(64), torch.full((T,), -1, dtype=torch.int32, device="cuda")
    keep[1], keep[17] = 510, 36
    ws = _ws(cache, s, e, H)

    def step():
        dv.dv_kv_append(cache, 0, s, e, qkv[:, H:2 * H], qkv[:, 2 * H:], q=qkv[:, :H], q_out=q, rope=rope)
        dv.dv_tree_attention(cache, 0, s, e, q, out, 0.125, ws)
        dv.dv_prompt_attention(cache, 0, s, e, q, out, 0.125, ws)
        dv.dv_kv_compact(cache, 0, 1, s, e, keep)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        first = (out.clone(), K.clone(), V.clone())
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in (out, K[0, :, :, :, 500:], V[0, :, :, 500:]):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0])
    for b, _, a, z in R.spans(s, e):
        assert torch.equal(K[0, b, :, :, a:z], first[1][0, b, :, :, a:z])
        assert torch.equal(V[0, b, :, a:z], first[2][0, b, :, a:z])
    qkv.normal_(generator=gen)
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(out, replayed) and not torch.equal(out, first[0])


def test_gpu_refusals():
    gen = _gen(1)
    cache, K, V = R.make_cache("fp16", 1, 1, 2, 64, 64, gen)
    s, e = np.array([0], np.int32), np.array([8], np.int32)
    q = torch.zeros(8, 2, 64, dtype=torch.float16, device="cuda")
    o = torch.zeros_like(q)

    def status(fn):
        with pytest.raises(dv.DvError) as ei:
            fn()
        return ei.value.status

    assert status(lambda: dv.dv_prompt_attention(cache, 0, s, e, q, q, 0.125, _ws(cache, s, e, 2))) == \
        dv.DV_ERR_INVALID_ARG  # out overlaps q
    assert status(lambda: dv.dv_kv_append(cache, 0, s, e, q, o, q=q, q_out=q)) == dv.DV_ERR_INVALID_ARG
    host = torch.zeros(8, 2, 64, dtype=torch.float16).pin_memory()
    assert status(lambda: dv.dv_prompt_attention(cache, 0, s, e, host, o, 0.125, _ws(cache, s, e, 2))) == \
        dv.DV_ERR_INVALID_ARG
    odd = torch.zeros(8 * 128 + 8, dtype=torch.float16, device="cuda")[4:8 * 128 + 4].view(8, 2, 64)
    assert status(lambda: dv.dv_prompt_attention(cache, 0, s, e, odd, o, 0.125, _ws(cache, s, e, 2))) == \
        dv.DV_ERR_MISALIGNED
    skew = torch.zeros(8, 2 * 64 + 4, dtype=torch.float16, device="cuda")[:, :128].view(8, 2, 64)
    assert status(lambda: dv.dv_prompt_attention(cache, 0, s, e, skew, o, 0.125, _ws(cache, s, e, 2))) == \
        dv.DV_ERR_MISALIGNED
    need = dv.dv_attention_workspace(cache, s, e, 2)
    if need:
        small = torch.zeros(need - 16, dtype=torch.uint8, device="cuda")
        assert status(lambda: dv.dv_prompt_attention(cache, 0, s, e, q, o, 0.125, small)) == \
            dv.DV_ERR_BUFFER_TOO_SMALL
    torch.cuda.synchronize()


def test_outputs_and_workspace_on_the_cache_are_refused():
    """What a call writes besides its rows shares no bytes with the layer it
    reads (another layer's are the caller's business), nor with the tree."""
    cache, K, V = R.make_cache("fp16", 2, 1, 2, 64, 4096, _gen(2))
    before = K.clone(), V.clone()
    s, e = np.array([0], np.int32), np.array([8], np.int32)
    q = torch.zeros(8, 2, 64, dtype=torch.float16, device="cuda")
    o, ws = torch.zeros_like(q), _ws(cache, s, e, 2)
    tree = torch.full((8,), 255, dtype=torch.int64, device="cuda")

    def refused(fn):
        with pytest.raises(dv.DvError) as ei:
            fn()
        assert ei.value.status == dv.DV_ERR_INVALID_ARG and "overlaps" in str(ei.value)

    for t in (K, V):
        on = t[1].reshape(-1)[:8 * 128].view(8, 2, 64)
        refused(lambda: dv.dv_kv_append(cache, 1, s, e, q, q, q=q, q_out=on))
        refused(lambda: dv.dv_prompt_attention(cache, 1, s, e, q, on, 0.125, ws))
        refused(lambda: dv.dv_tree_attention(cache, 1, s, e, q, on, 0.125, ws, tree=tree))
        refused(lambda: dv.dv_prompt_attention(cache, 1, s, e, q, o, 0.125, t[1].reshape(-1)))
    bits = o.view(-1).view(torch.int64)[:8]
    refused(lambda: dv.dv_tree_attention(cache, 0, s, e, q, o, 0.125, ws, tree=bits))
    refused(lambda: dv.dv_tree_attention(cache, 0, s, e, q, o, 0.125, ws, tree=ws.view(torch.int64)[:8]))
    torch.cuda.synchronize()
    assert torch.equal(K, before[0]) and torch.equal(V, before[1])


# ---- compact ---------------------------------------------------------------------------

@pytest.mark.parametrize("P", [1, 2, 4])
@pytest.mark.parametrize("B, H, D, S, L", [(2, 3, 64, 200, 2), (1, 1, 16, 3000, 1), (3, 2, 128, 90, 3),
                                           (40, 1, 32, 40, 1), (1, 2, 80, 1500, 1), (1, 1, 384, 700, 1)])
def test_compact(P, B, H, D, S, L):
    """Every row of the range from its list entry as the cache was, whatever
    the list overlaps; entries out of place leave their rows."""
    x = 16 // P
    rng = np.random.default_rng(S + P)
    n = B * H * D * S
    stride = n + 16
    k = torch.randint(0, 256, (L, stride * P), dtype=torch.uint8, device="cuda")
    v = torch.randint(0, 256, (L, stride * P), dtype=torch.uint8, device="cuda")
    cache = dv.Cache(L, B, H, D, S, P, k, v, layer_stride_elems=stride)
    K = k[:, :n * P].view(L, B, H, D // x, S, 16)
    V = v[:, :n * P].view(L, B, H, S, D * P)
    s = rng.integers(0, S // 3, size=B).astype(np.int32)
    e = s + rng.integers(0, S // 2 + 1, size=B).astype(np.int32)
    keep = []
    for a, z in zip(s.tolist(), e.tolist()):
        m = z - a
        kind = rng.integers(0, 3)
        if kind == 0:    # any rows at or past their destination, in any order
            rows = [int(rng.integers(a + i, S)) for i in range(m)]
        elif kind == 1:  # ascending (an eviction)
            rows = sorted(rng.choice(np.arange(a, S), size=m, replace=False).tolist())
        else:            # with entries that are out of place
            rows = [int(rng.choice([-1, S, S + 5, a - 1, -2 ** 31, a + i, S - 1])) for i in range(m)]
        keep += rows
    l0, l1 = (1, L) if L > 1 else (0, 1)
    wk, wv = K.clone(), V.clone()
    for b, t, a, z in R.spans(s, e):
        for i, src in enumerate(keep[t:t + z - a]):
            if a + i <= src < S:
                wk[l0:l1, b, :, :, a + i] = K[l0:l1, b, :, :, src]
                wv[l0:l1, b, :, a + i] = V[l0:l1, b, :, src]
    dv.dv_kv_compact(cache, l0, l1, s, e, torch.tensor(keep, dtype=torch.int32, device="cuda"))
    assert torch.equal(K, wk) and torch.equal(V, wv)

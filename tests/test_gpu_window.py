"""dv_window_attention against its plain 64-bit form (tests/bounded_refs.py derives the
bounds): types, head layouts, odd sizes, windows and first rows that end inside tiles or pass
the sequence, values that a mask hides, streams, graphs."""
import math

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv
from tests import bounded_refs as W
from tests import operator_refs as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    dv.dv_attention_check()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ws(cache, s, e, heads):
    """The workspace, filled with NaN bits: it needs no initial value."""
    n = dv.dv_attention_workspace(cache, s, e, heads)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None


def _attend(cache, layer, s, e, q, scale, window, sinks, out=None, stream=None):
    out = torch.full_like(q, math.nan) if out is None else out
    dv.dv_window_attention(cache, layer, s, e, q, out, scale, window, sinks, _ws(cache, s, e, q.shape[1]), stream=stream)
    return out


def _hide(K, V, s, e, window, sinks):
    """NaN, infinities and huge values in every row that no token attends, and past the rows."""
    for b, _, a, z in R.spans(s, e):
        seen = torch.zeros(K.shape[4], dtype=torch.bool, device="cuda")
        if z > a:
            seen[:z] = W.window_mask(a, z, window, sinks).any(0)
        bad = torch.tensor([math.nan, math.inf, -math.inf, 6e4], device="cuda", dtype=K.dtype)
        for t, dim in ((K[:, b], 3), (V[:, b], 2)):
            at = (~seen).nonzero().flatten()
            fill = bad[at % 4].view([-1 if i == dim else 1 for i in range(t.dim())])
            t.index_copy_(dim, at, fill.expand([len(at) if i == dim else x for i, x in enumerate(t.shape)]).contiguous())


CASES = [
    # B, H, G, D, S, ctx, new, window, sinks
    (1, 1, 1, 64, 1, (0, 0), (1, 1), 1, 0),
    (2, 2, 1, 64, 300, (0, 299), (1, 1), 1, 0),
    (3, 2, 1, 128, 700, (100, 690), (1, 1), 128, 4),
    (3, 2, 4, 128, 1024, (0, 1000), (1, 9), 200, 1),
    (2, 2, 8, 64, 2000, (900, 1900), (1, 16), 257, 130),
    (2, 1, 71, 64, 400, (0, 390), (1, 3), 33, 5),
    (1, 1, 128, 128, 500, (400, 440), (33, 33), 100, 128),
    (2, 3, 1, 64, 1300, (0, 100), (600, 1200), 128, 0),
    (2, 2, 1, 128, 1500, (0, 0), (1, 1500), 500, 4),
    (3, 2, 3, 64, 421, (0, 100), (0, 321), 60, 16),
    (2, 2, 2, 8, 1024, (512, 600), (300, 400), 96, 96),
    (2, 2, 1, 72, 517, (0, 129), (250, 388), 129, 127),      # an odd S: rows of one chunk a run
    (2, 1, 5, 96, 1261, (900, 900), (200, 255), 300, 301),
    (2, 1, 2, 120, 2000, (1500, 1700), (255, 256), 1000, 513),
    (36, 2, 1, 64, 200, (0, 120), (0, 60), 40, 3),
    (1, 2, 1, 128, 4096, (2048, 2048), (2048, 2048), 1024, 16),
    (1, 1, 2, 64, 20000, (19500, 19500), (300, 300), 4096, 4),
    (1, 2, 4, 128, 30000, (29000, 29900), (1, 1), 20000, 64),  # cut among many CTAs
    (4, 64, 1, 128, 1500, (600, 900), (40, 600), 333, 7),       # more units than SMs
    (5, 70, 1, 128, 1200, (0, 1130), (1, 20), 100, 4),
    # many units of few rows: two heads at a time, an odd number of them, cut among CTAs
    (11, 71, 1, 128, 700, (0, 690), (1, 3), 200, 4),
    (10, 63, 4, 64, 500, (300, 480), (0, 16), 130, 33),
    (310, 2, 2, 40, 321, (0, 300), (1, 5), 64, 0),
    (3, 301, 1, 72, 900, (800, 899), (1, 1), 700, 100),
    (2, 2, 1, 64, 900, (300, 400), (1, 400), 900, 0),           # windows that hide nothing
    (2, 2, 2, 128, 900, (300, 400), (1, 64), 50, 900),          # first rows that hide nothing
    (1, 1, 1, 64, 257, (0, 0), (257, 257), 1, 1),
    (2, 1, 1, 128, 1024, (1000, 1000), (24, 24), 2**31 - 1, 2**31 - 1),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B, H, G, D, S, ctx, new, window, sinks", CASES)
def test_window_attention(dtype, B, H, G, D, S, ctx, new, window, sinks):
    rng = np.random.default_rng(S + window)
    gen = _gen(S + D)
    s = rng.integers(ctx[0], ctx[1] + 1, size=B).astype(np.int32)
    n = rng.integers(new[0], new[1] + 1, size=B).astype(np.int32)
    if new[0] == 0 and B > 1:
        n[rng.integers(B)] = 0
    e = (s + np.minimum(n, S - s)).astype(np.int32)
    cache, K, V = R.make_cache(dtype, 2, B, H, D, S, gen)
    q = torch.empty(int((e - s).sum()), H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) * 2
    scale = D ** -0.5
    want, tol, _, _ = W.attend_ref(K[1], V[1], s, e, q, scale, window, sinks)
    _hide(K, V, s, e, window, sinks)
    got = _attend(cache, 1, s, e, q, scale, window, sinks)
    R.assert_within(got, want, tol)
    assert torch.equal(_attend(cache, 1, s, e, q, scale, window, sinks), got)  # the same bits again


def test_a_window_of_every_row_is_causal_attention():
    gen = _gen(5)
    s, e = np.array([0, 40, 300], np.int32), np.array([200, 41, 500], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 3, 2, 64, 512, gen)
    q = torch.empty(401, 4, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    want = torch.empty_like(q)
    dv.dv_prompt_attention(cache, 0, s, e, q, want, 0.125, _ws(cache, s, e, 4))
    for window, sinks in ((512, 0), (500, 0), (1, 512), (10**9, 3)):
        assert torch.equal(_attend(cache, 0, s, e, q, 0.125, window, sinks), want)


@pytest.mark.parametrize("seed", range(24))
def test_random_windows(seed):
    rng = np.random.default_rng(seed)
    gen = _gen(seed)
    dtype = ["fp16", "bf16"][rng.integers(2)]
    B, H, G, D = int(rng.integers(1, 9)), int(rng.integers(1, 9)), int(rng.integers(1, 9)), 8 * int(rng.integers(1, 17))
    s = rng.integers(0, int(rng.choice([1, 200, 3000])), size=B).astype(np.int32)
    e = s + rng.integers(0, int(rng.choice([2, 5, 60, 700])), size=B).astype(np.int32)
    window, sinks = int(np.exp(rng.uniform(0, 8))), int(rng.choice([0, 1, 4, 31, 128, 300]))
    S = int(e.max()) + int(rng.integers(0, 9)) + 1
    cache, K, V = R.make_cache(dtype, 1, B, H, D, S, gen)
    wide = torch.empty(int((e - s).sum()), H * G * D + 24, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    q = wide[:, 8:8 + H * G * D].view(-1, H * G, D)  # strided tokens
    want, tol, _, _ = W.attend_ref(K[0], V[0], s, e, q, 0.2, window, sinks)
    _hide(K, V, s, e, window, sinks)
    out = torch.full((len(q) + 2, H * G, D), math.nan, dtype=q.dtype, device="cuda")
    _attend(cache, 0, s, e, q, 0.2, window, sinks, out=out[1:-1] if len(q) else out[:0])
    R.assert_within(out[1:-1], want, tol)
    assert bool(torch.isnan(out[0]).all() and torch.isnan(out[-1]).all())  # what lies around it is as it was


TREES = [
    # B, H, G, D, S, ctx, new, window, sinks
    (3, 2, 1, 128, 700, (0, 630), (1, 9), 64, 4),
    (3, 2, 4, 128, 1000, (100, 936), (1, 64), 100, 0),
    (2, 2, 8, 64, 2000, (1500, 1900), (33, 64), 257, 130),
    (2, 1, 71, 64, 400, (0, 390), (1, 3), 80, 5),
    (2, 1, 128, 128, 500, (400, 430), (64, 64), 64, 1),      # windows that end among the new rows
    (3, 2, 3, 40, 260, (0, 140), (1, 64), 65, 0),
    (2, 2, 1, 72, 517, (200, 400), (1, 64), 1000, 3),         # windows that hide nothing
    (11, 71, 1, 128, 700, (0, 600), (1, 3), 200, 4),          # two heads at a time
    (10, 63, 4, 64, 500, (300, 480), (0, 16), 130, 33),
    (1, 2, 4, 128, 30000, (29000, 29900), (31, 31), 20000, 64),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B, H, G, D, S, ctx, new, window, sinks", TREES)
def test_window_over_trees(dtype, B, H, G, D, S, ctx, new, window, sinks):
    """Drafted tokens: the new rows of their bits, and of the rows before those within the window that
    ends at their depth; a token without any bits too."""
    rng = np.random.default_rng(S + window)
    gen = _gen(S + D)
    s = rng.integers(ctx[0], ctx[1] + 1, size=B).astype(np.int32)
    n = rng.integers(new[0], new[1] + 1, size=B).astype(np.int32)
    e = (s + np.minimum(n, S - s)).astype(np.int32)
    cache, K, V = R.make_cache(dtype, 1, B, H, D, S, gen)
    bits, masks = [], []
    for a, z in zip(s.tolist(), e.tolist()):
        m = z - a
        own = R.random_tree(m, rng)[0]
        if m > 2:
            own[m // 2] = 0
        at = torch.tensor([a + max(x.bit_count() - 1, 0) for x in own], device="cuda")[:, None]
        j = torch.arange(z, device="cuda")
        ok = ((j < a) & ((j > at - window) | (j < sinks)))
        for i, x in enumerate(own):
            for k in range(m):
                ok[i, a + k] = bool(x >> k & 1)
        masks.append(ok)
        bits += own
    q = torch.empty(int((e - s).sum()), H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) * 2
    want, tol, _, _ = W.attend_ref(K[0], V[0], s, e, q, 0.1, masks=masks)
    for b, (a, z) in enumerate(zip(s.tolist(), e.tolist())):  # garbage where no token looks
        hidden = torch.ones(S, dtype=torch.bool, device="cuda")
        hidden[:z] = ~masks[b].any(0) if z > a else True
        K[0, b].masked_fill_(hidden[None, None, :, None], math.nan)
        V[0, b].masked_fill_(hidden[None, :, None], math.inf)
    out = torch.full_like(q, math.nan)
    tree = R.bits_tensor(bits)
    dv.dv_window_attention(cache, 0, s, e, q, out, 0.1, window, sinks, _ws(cache, s, e, H * G), tree=tree)
    R.assert_within(out, want, tol)


def test_values_that_are_not_finite_reach_the_tokens_that_attend_them_alone():
    """An infinity in the first rows, a NaN at a window's edge: for each token as its row says."""
    gen = _gen(9)
    s, e = np.array([1000], np.int32), np.array([1140], np.int32)
    for window, sinks, rows in ((100, 4, (2, 3, 4, 905, 960, 1041, 1100)), (700, 130, (129, 130, 131, 301, 400, 1000))):
        cache, K, V = R.make_cache("bf16", 1, 1, 2, 64, 1200, gen)
        for i, r in enumerate(rows):
            V[0, 0, i % 2, r, 7 * i % 64] = (math.inf, math.nan, -math.inf)[i % 3]
        q = torch.empty(140, 6, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        want, tol, _, _ = W.attend_ref(K[0], V[0], s, e, q, 0.125, window, sinks)
        assert bool(want.isnan().any()) and bool(want.isfinite().any())
        R.assert_within(_attend(cache, 0, s, e, q, 0.125, window, sinks), want, tol)


def test_window_in_a_graph_on_a_side_stream():
    gen = _gen(11)
    s, e = np.array([700, 0], np.int32), np.array([701, 300], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 2, 4, 128, 1024, gen)
    q = torch.empty(301, 8, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    out, ws = torch.zeros_like(q), _ws(cache, s, e, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dv.dv_window_attention(cache, 0, s, e, q, out, 0.1, 130, 5, ws, stream=side)
    for _ in range(3):
        q.normal_(generator=gen)
        K.normal_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        want, tol, _, _ = W.attend_ref(K[0], V[0], s, e, q, 0.1, 130, 5)
        R.assert_within(out, want, tol)


def test_a_wait_that_gives_up_is_reported():
    gen = _gen(12)
    s, e = np.array([0], np.int32), np.array([700], np.int32)
    cache, K, V = R.make_cache("fp16", 1, 1, 2, 64, 700, gen)
    q = torch.empty(700, 2, 64, dtype=torch.float16, device="cuda").normal_(generator=gen)
    dv.dv_attention_check()
    dv.dv_debug_attention_tries(0)
    try:
        _attend(cache, 0, s, e, q, 0.125, 100, 4)
        with pytest.raises(dv.DvError) as ei:
            dv.dv_attention_check()
        assert ei.value.status == dv.DV_ERR_TIMEOUT
    finally:
        dv.dv_debug_attention_tries()
    want, tol, _, _ = W.attend_ref(K[0], V[0], s, e, q, 0.125, 100, 4)
    R.assert_within(_attend(cache, 0, s, e, q, 0.125, 100, 4), want, tol)

"""dv_kv_evict against a sort (tests/bounded_refs.py): which rows stay, ties, NaN and zeros,
and every byte of K, V and the weights; then the operators that bound a cache together."""
import math

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv
from tests import bounded_refs as W
from tests import operator_refs as R

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


INT = {1: torch.uint8, 2: torch.int16, 4: torch.int32}


def _cache(L, B, H, D, S, P, gen, gap=0):
    stride = B * H * D * S + gap
    k, v = (torch.randint(0, 250, (L, stride), generator=gen, device="cuda").to(INT[P]) for _ in range(2))
    for t in (k, v):
        t.random_(generator=gen)
    n, x = B * H * D * S, 16 // P
    return (dv.Cache(L, B, H, D, S, P, k, v, layer_stride_elems=stride), k[:, :n].view(L, B, H, D // x, S, x),
            v[:, :n].view(L, B, H, S, D), k, v)


def _weights(kind, shape, gen):
    x = torch.rand(shape, generator=gen, device="cuda")
    if kind == "few":  # few rows with much
        return x ** 8 * 30
    if kind == "ties":
        return (x * 5).floor() / 4
    if kind == "zero":
        return torch.zeros_like(x)
    if kind == "signs":  # what no sum of weights is, but a user's own scores may be
        y = (x * 7).floor() - 3
        y[x < 0.1] = -0.0
        y[(x > 0.2) & (x < 0.3)] = math.nan
        y[(x > 0.3) & (x < 0.32)] = -math.nan
        y[(x > 0.4) & (x < 0.45)] = math.inf
        y[(x > 0.5) & (x < 0.55)] = -math.inf
        y[(x > 0.6) & (x < 0.65)] *= 1e-42
        return y
    return x


def _check(cache, K, V, k, v, l0, l1, rows, kept, sinks, recent, mass, in_place, stream=None):
    B, H, S = K.shape[1], K.shape[2], K.shape[4]
    T = int(kept.sum())
    lists = W.evict_rows(mass, rows, kept, sinks, recent)
    k0, v0, K0, V0, m0 = k.clone(), v.clone(), K.clone(), V.clone(), mass.clone()
    out = mass if in_place else torch.full_like(mass, -7.0)
    want = out.clone()
    keep = torch.full((l1 - l0, H, T + 0), -1, dtype=torch.int32, device="cuda")
    dv.dv_kv_evict(cache, l0, l1, rows, kept, sinks, recent, mass, keep, mass_out=None if in_place else out, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(keep.cpu(), torch.tensor([[sum(x, []) for x in y] for y in lists],
                                                dtype=torch.int32).view(l1 - l0, H, T))
    for l in range(l1 - l0):
        for h in range(H):
            for b, (n, m) in enumerate(zip(rows.tolist(), kept.tolist())):
                at = torch.tensor(lists[l][h][b], dtype=torch.int64, device="cuda")
                K0[l0 + l, b, h, :, :m] = K0[l0 + l, b, h][:, at]
                V0[l0 + l, b, h, :m] = V0[l0 + l, b, h][at]
                want[l, b, h, :m] = m0[l, b, h][at]
                want[l, b, h, m:n] = 0.0
    assert torch.equal(K, K0) and torch.equal(V, V0)
    assert torch.equal(out.view(torch.int32), want.view(torch.int32))
    if not in_place:
        assert torch.equal(mass.view(torch.int32), m0.view(torch.int32))
    n = K[0].numel()  # what lies between the layers
    assert torch.equal(k[:, n:], k0[:, n:]) and torch.equal(v[:, n:], v0[:, n:])


CASES = [
    # L, B, H, D, S, P, rows, kept, sinks, recent, kind
    (1, 1, 1, 8, 2, 2, [2], [1], 0, 0, "plain"),
    (1, 1, 1, 64, 1, 2, [1], [0], 0, 0, "plain"),            # everything goes
    (2, 3, 2, 64, 40, 2, [40, 7, 0], [9, 7, 0], 2, 3, "few"),  # some keep all, one has none
    (1, 2, 3, 64, 433, 2, [433, 401], [400, 400], 4, 100, "few"),
    (2, 2, 5, 128, 600, 2, [599, 520], [300, 257], 4, 128, "ties"),
    (1, 2, 2, 128, 600, 2, [600, 600], [100, 300], 0, 0, "zero"),    # the lowest rows stay
    (1, 2, 4, 64, 700, 2, [700, 650], [350, 64], 3, 30, "signs"),
    (1, 1, 2, 64, 700, 2, [700], [20], 10, 10, "plain"),       # no room between the first and the last
    (1, 1, 2, 64, 700, 2, [700], [699], 0, 699, "plain"),
    (1, 1, 2, 64, 700, 2, [700], [699], 699, 0, "plain"),
    (3, 40, 2, 32, 30, 4, [30] * 20 + [17] * 20, [11] * 30 + [17] * 10, 1, 2, "ties"),
    (1, 2, 2, 16, 300, 1, [300, 10], [77, 9], 1, 1, "few"),
    (1, 1, 3, 72, 513, 2, [511], [256], 4, 0, "few"),
    (1, 1, 1, 320, 300, 4, [300], [100], 1, 5, "plain"),       # more chunks than a slice
    (2, 1, 2, 64, 5000, 2, [4999], [2500], 16, 512, "few"),
    (1, 1, 2, 128, 40000, 2, [39999], [5000], 4, 1000, "few"),
    (1, 2, 1, 64, 9000, 2, [8999, 8192], [8998, 100], 4, 0, "ties"),
    (1, 2, 2, 128, 30000, 2, [29999, 20000], [5000, 19999], 4, 1000, "ties"),
    (1, 1, 1, 16, 420000, 2, [419999], [2000], 4, 100, "few"), 
    (1, 2, 1, 16, 420000, 2, [419999, 300], [2000, 300], 4, 100, "ties"),
    (8, 4, 40, 64, 200, 2, [200, 150, 199, 60], [100, 60, 198, 60], 4, 16, "few"),
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("L, B, H, D, S, P, rows, kept, sinks, recent, kind", CASES)
def test_evict(L, B, H, D, S, P, rows, kept, sinks, recent, kind, in_place):
    gen = _gen(S + L)
    cache, K, V, k, v = _cache(L, B, H, D, S, P, gen, gap=64)
    mass = _weights(kind, (L, B, H, S), gen)
    _check(cache, K, V, k, v, 0, L, np.array(rows, np.int32), np.array(kept, np.int32), sinks, recent, mass, in_place)


@pytest.mark.parametrize("seed", range(24))
def test_random_evictions(seed):
    rng = np.random.default_rng(seed)
    gen = _gen(seed)
    L, B, H, D = int(rng.integers(1, 4)), int(rng.integers(1, 6)), int(rng.integers(1, 6)), 16 * int(rng.integers(1, 10))
    S = int(np.exp(rng.uniform(0.7, 8.3)))
    rows = rng.integers(0, S + 1, size=B).astype(np.int32)
    kept = (rows * rng.choice([0.1, 0.5, 0.9, 1.0], size=B)).astype(np.int32)
    least = int(kept[kept < rows].min()) if bool((kept < rows).any()) else 4
    sinks = int(rng.integers(0, least // 2 + 1))
    recent = int(rng.integers(0, least - sinks + 1))
    l0 = int(rng.integers(0, L))
    l1 = int(rng.integers(l0 + 1, L + 1))
    cache, K, V, k, v = _cache(L, B, H, D, S, int(rng.choice([1, 2, 4])), gen, gap=int(rng.choice([0, 16])))
    mass = _weights(str(rng.choice(["plain", "few", "ties", "zero", "signs"])), (l1 - l0, B, H, S), gen)
    _check(cache, K, V, k, v, l0, l1, rows, kept, sinks, recent, mass, bool(rng.integers(2)))


UNTOUCHED = [
    # L, B, H, D, S, rows, kept: sequences that keep all beside others that give rows up
    (1, 2, 2, 16, 420000, [420000, 600], [420000, 300]),
    (1, 3, 1, 64, 30000, [700, 29999, 650], [350, 29999, 64]),
    (2, 2, 1, 64, 9000, [8999, 8192], [8999, 8192]),
    (1, 2, 1, 64, 17000, [16999, 9000], [16999, 1000]),
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("L, B, H, D, S, rows, kept", UNTOUCHED)
def test_long_sequences_that_keep_all_beside_short_ones(L, B, H, D, S, rows, kept, in_place):
    gen = _gen(S)
    cache, K, V, k, v = _cache(L, B, H, D, S, 2, gen, gap=16)
    mass = _weights("signs", (L, B, H, S), gen)
    _check(cache, K, V, k, v, 0, L, np.array(rows, np.int32), np.array(kept, np.int32), 4, 20, mass, in_place)


def test_sequences_that_keep_all_do_not_choose_the_kernel():
    """More rows than a cluster's shared memory holds weights of, none of which is searched: the
    short sequence's weights are held in shared memory all the same."""
    from torch.profiler import ProfilerActivity, profile

    gen = _gen(9)
    cache, _, _, _, _ = _cache(1, 2, 1, 16, 420000, 2, gen)
    mass = _weights("few", (1, 2, 1, 420000), gen)
    keep = torch.empty(1, 1, 420300, dtype=torch.int32, device="cuda")
    rows, kept = np.array([420000, 600], np.int32), np.array([420000, 300], np.int32)
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]):  # (a process's first recording may miss kernels)
        keep.zero_()
        torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        dv.dv_kv_evict(cache, 0, 1, rows, kept, 4, 20, mass, keep)
        torch.cuda.synchronize()
    names = [e.name for e in prof.events() if "evict_kernel" in e.name]
    if not names:
        pytest.skip("the profiler records no kernels here")
    assert len(names) == 1 and "true>" in names[0], names


def test_nothing_to_do():
    gen = _gen(3)
    cache, K, V, k, v = _cache(2, 2, 2, 64, 50, 2, gen)
    mass = _weights("plain", (2, 2, 2, 50), gen)
    full = np.array([50, 20], np.int32)
    _check(cache, K, V, k, v, 0, 2, full, full, 30, 30, mass, True)
    none = np.zeros(2, np.int32)
    _check(cache, K, V, k, v, 0, 2, none, none, 0, 0, mass, True)
    dv.dv_kv_evict(cache, 1, 1, full, full, 0, 0, mass[:0], torch.empty(0, dtype=torch.int32, device="cuda"))


def test_evict_in_a_graph_on_a_side_stream():
    gen = _gen(4)
    cache, K, V, k, v = _cache(1, 2, 4, 64, 500, 2, gen)
    rows, kept = np.array([500, 300], np.int32), np.array([200, 150], np.int32)
    mass, out = _weights("few", (1, 2, 4, 500), gen), torch.zeros(1, 2, 4, 500, device="cuda")
    keep = torch.zeros(1, 4, 350, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dv.dv_kv_evict(cache, 0, 1, rows, kept, 4, 50, mass, keep, mass_out=out, stream=side)
    for _ in range(3):
        mass.copy_(_weights("ties", mass.shape, gen))
        K.random_(generator=gen)
        K0, lists = K.clone(), W.evict_rows(mass, rows, kept, 4, 50)
        graph.replay()
        torch.cuda.synchronize()
        assert keep[0].tolist() == [sum(x, []) for x in lists[0]]
        for h in range(4):
            for b, m in enumerate(kept.tolist()):
                assert torch.equal(K[0, b, h, :, :m], K0[0, b, h][:, torch.tensor(lists[0][h][b], device="cuda")])


def test_two_evictions_in_flight_on_two_streams_and_a_captured_one():
    """Clusters (two long sequences) and single CTAs at once, eager and replayed."""
    gen = _gen(8)
    jobs = []
    for L, B, H, S, rows, kept in ((1, 1, 2, 30000, [29000], [4000]), (4, 4, 20, 300, [300, 200, 150, 299], [90] * 4)):
        cache, K, V, k, v = _cache(L, B, H, 64, S, 2, gen)
        mass = _weights("few", (L, B, H, S), gen)
        rows, kept = np.array(rows, np.int32), np.array(kept, np.int32)
        keep = torch.zeros(L, H, int(kept.sum()), dtype=torch.int32, device="cuda")
        out = torch.zeros_like(mass)
        jobs.append((cache, K, V, K.clone(), V.clone(), mass, out, rows, kept, keep, torch.cuda.Stream(), torch.cuda.CUDAGraph()))
    def check():
        torch.cuda.synchronize()
        for cache, K, V, K0, V0, mass, out, rows, kept, keep, _, _ in jobs:
            lists = W.evict_rows(mass, rows, kept, 4, 20)
            assert keep.tolist() == [[sum(x, []) for x in y] for y in lists]
            for l, h, b in ((0, 0, 0), (K.shape[0] - 1, K.shape[2] - 1, K.shape[1] - 1)):
                at = torch.tensor(lists[l][h][b], device="cuda")
                assert torch.equal(K[l, b, h, :, :kept[b]], K0[l, b, h][:, at])
                assert torch.equal(V[l, b, h, :kept[b]], V0[l, b, h][at])
                assert torch.equal(out[l, b, h, :kept[b]], mass[l, b, h][at])
            K.copy_(K0)
            V.copy_(V0)
            keep.zero_()
        torch.cuda.synchronize()
    def call(j):
        cache, _, _, _, _, mass, out, rows, kept, keep, stream, _ = j
        dv.dv_kv_evict(cache, 0, cache.num_layers, rows, kept, 4, 20, mass, keep, mass_out=out, stream=stream)
    torch.cuda.synchronize()
    for j in jobs:
        call(j)
    check()
    for j in jobs:
        with torch.cuda.graph(j[-1], stream=j[-2]):
            call(j)
    for _ in range(2):
        for j in jobs:
            with torch.cuda.stream(j[-2]):
                j[-1].replay()
        check()


@pytest.mark.parametrize("fresh", [False, True])
def test_an_evicted_cache_and_its_replica(fresh):
    """A replica's records hold rows as they were.  After an eviction a record of [0, kept) goes to
    the log (or, `fresh`, is the first of an emptied one) and the deltas go on; a restore gives every
    row in use, from where the kept weights choose the same rows again.  Without that record the
    restore brings given-up rows back."""
    gen = _gen(12)
    L, B, H, D, S, P = 2, 3, 3, 64, 120, 2
    cache, K, V, k, v = _cache(L, B, H, D, S, P, gen)
    mass = _weights("few", (L, B, H, S), gen)
    used, zero = np.array([80, 33, 100], np.int32), np.zeros(B, np.int32)
    kept = np.array([40, 33, 52], np.int32)

    def arena():
        return torch.empty(L * B * H * D * S * P * 8, dtype=torch.uint8).pin_memory()

    rep, bare = (dv.Replica(arena(), B) for _ in range(2))
    step = 0

    def record(logs, s, e):
        nonlocal step
        for r in logs:
            r.append(cache, 0, L, s, e, step)
        step += 1

    def decode(logs, steps):
        nonlocal used
        for _ in range(steps):
            for b in range(B):
                K[:, b, :, :, used[b]].random_(generator=gen)
                V[:, b, :, used[b]].random_(generator=gen)
                mass[:, b, :, used[b]] = torch.rand(L, H, generator=gen, device="cuda")
            record(logs, used, used + 1)
            used = (used + 1).astype(np.int32)

    def restored(r, batched):
        back, BK, BV, bk, bv = _cache(L, B, H, D, S, P, gen)
        (r.restore_batched if batched else r.restore)(back)
        torch.cuda.synchronize()
        same = all(torch.equal(BK[:, b, :, :, :n], K[:, b, :, :, :n]) and torch.equal(BV[:, b, :, :n], V[:, b, :, :n])
                   for b, n in enumerate(used.tolist()))
        return same, (back, BK, BV)

    record((rep, bare), zero, used)
    decode((rep, bare), 5)
    assert restored(rep, True)[0]
    keep = torch.empty(L, H, int(kept.sum()), dtype=torch.int32, device="cuda")
    dv.dv_kv_evict(cache, 0, L, used, kept, 4, 8, mass, keep)
    used = kept
    torch.cuda.synchronize()
    if fresh:
        rep.truncate(0)
        assert rep.info() == (0, 0)
    record((rep,), zero, kept)
    decode((rep, bare), 4)
    torch.cuda.synchronize()
    for batched in (False, True):
        same, (back, BK, BV) = restored(rep, batched)
        assert same
        assert not restored(bare, batched)[0]
    again, lists = np.array([20, 37, 30], np.int32), []
    for c in (cache, back):
        keep = torch.empty(L, H, int(again.sum()), dtype=torch.int32, device="cuda")
        dv.dv_kv_evict(c, 0, L, used, again, 4, 8, mass, keep, mass_out=torch.empty_like(mass))
        lists.append(keep)
    assert torch.equal(*lists)
    for b, n in enumerate(again.tolist()):
        assert torch.equal(BK[:, b, :, :, :n], K[:, b, :, :, :n]) and torch.equal(BV[:, b, :, :n], V[:, b, :, :n])


def test_a_cache_past_2_31_elements():
    """The last head of a layer of 2^31 elements: rows far apart moved to its front."""
    B, H, D, S = 2, 64, 128, 131072
    k, v = (torch.zeros(B * H * D * S, dtype=torch.int16, device="cuda") for _ in range(2))
    cache = dv.Cache(1, B, H, D, S, 2, k, v)
    K, V = k.view(1, B, H, D // 8, S, 8), v.view(1, B, H, S, D)
    mass = torch.zeros(1, B, H, S, device="cuda")
    mass[0, 1, 63, [5, 100000, 131071]] = 1.0
    for i, r in enumerate((5, 100000, 131071)):
        K[0, 1, 63, :, r] = i + 1
        V[0, 1, 63, r] = i + 1
    rows, kept = np.array([0, S], np.int32), np.array([0, 3], np.int32)
    keep = torch.zeros(1, H, 3, dtype=torch.int32, device="cuda")
    dv.dv_kv_evict(cache, 0, 1, rows, kept, 0, 0, mass, keep)
    assert keep[0, 63].tolist() == [5, 100000, 131071] and keep[0, 62].tolist() == [0, 1, 2]
    assert K[0, 1, 63, :, :4].amin((0, 2)).tolist() == [1, 2, 3, 0] == V[0, 1, 63, :4].amin(1).tolist()
    assert mass[0, 1, 63, :4].tolist() == [1.0, 1.0, 1.0, 0.0] and float(mass.sum()) == 3.0


def test_a_bounded_cache_as_it_is_used():
    """Two layers decode in a cache of 96 rows a sequence: the prompt is scored, every layer evicts
    by itself down to 64 rows whenever some sequence has passed 90, the second layer's attention
    sees a window; against the same steps in 64 bits on the rows that the eviction kept."""
    gen = _gen(6)
    L, B, H, G, D, S, budget, sinks, recent = 2, 2, 2, 2, 64, 96, 64, 2, 8
    cache, K, V = R.make_cache("bf16", L, B, H, D, S, gen)
    mass = torch.zeros(L, B, H, S, device="cuda")
    shadow, stol = mass.double(), torch.zeros_like(mass, dtype=torch.float64)
    rope = dv.Rope(D)
    used, pos = np.zeros(B, np.int32), np.zeros(B, np.int32)
    evictions = 0
    for new in ([80, 30], *([1, 2] for _ in range(60))):
        n = np.array(new, np.int32)
        if int((used + n).max()) > 90:
            kept = np.minimum(used, budget).astype(np.int32)
            keep = torch.empty(L, H, int(kept.sum()), dtype=torch.int32, device="cuda")
            lists = W.evict_rows(mass, used, kept, sinks, recent)
            before = K.clone(), V.clone()
            dv.dv_kv_evict(cache, 0, L, used, kept, sinks, recent, mass, keep)
            for l in range(L):
                for h in range(H):
                    assert keep[l, h].tolist() == sum(lists[l][h], [])
                    for b in range(B):
                        at = torch.tensor(lists[l][h][b], device="cuda")
                        assert torch.equal(K[l, b, h, :, :kept[b]], before[0][l, b, h][:, at])
                        assert torch.equal(V[l, b, h, :kept[b]], before[1][l, b, h][at])
                        shadow[l, b, h, :kept[b]] = shadow[l, b, h][at]
                        shadow[l, b, h, kept[b]:] = 0
                        stol[l, b, h, :kept[b]] = stol[l, b, h][at]
                        stol[l, b, h, kept[b]:] = 0
            used, evictions = kept, evictions + 1
        e = (used + n).astype(np.int32)
        at = np.concatenate([p + np.arange(m) for p, m in zip(pos, n)]).astype(np.int32)
        for l in range(L):
            x = torch.empty(int(n.sum()), H * (G + 2), D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
            q = dv.dv_kv_append(cache, l, used, e, x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], q=x[:, :G * H],
                                rope=rope, positions=torch.from_numpy(at).cuda())
            out = torch.empty_like(q)
            ws = torch.empty(dv.dv_scored_attention_workspace(cache, used, e, G * H), dtype=torch.uint8, device="cuda")
            dv.dv_scored_attention(cache, l, used, e, q, out, 0.125, mass[l], ws, last=0 if new[0] == 1 else 32)
            want, tol, m, mtol = W.attend_ref(K[l], V[l], used, e, q, 0.125, last=0 if new[0] == 1 else 32,
                                              mass=shadow[l])
            R.assert_within(out, want, tol)
            stol[l] += mtol  # (the steps' errors add up)
            R.assert_within(mass[l], m, stol[l])
            shadow[l] = m
            if l == 1:
                dv.dv_window_attention(cache, l, used, e, q, out, 0.125, 24, sinks, ws)
                want, tol, _, _ = W.attend_ref(K[l], V[l], used, e, q, 0.125, 24, sinks)
                R.assert_within(out, want, tol)
        used, pos = e, pos + n
    assert evictions >= 2
    dv.dv_attention_check()

"""dv_scored_attention against its plain 64-bit form (tests/bounded_refs.py derives the
bounds): outputs and accumulated weights for types, head layouts, odd sizes, counted tokens,
values that a mask hides, streams, graphs."""
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
    n = dv.dv_scored_attention_workspace(cache, s, e, heads)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None


def _attend(cache, layer, s, e, q, scale, mass, last=0, out=None):
    out = torch.full_like(q, math.nan) if out is None else out
    dv.dv_scored_attention(cache, layer, s, e, q, out, scale, mass, _ws(cache, s, e, q.shape[1]), last=last)
    return out


def _check(cache, K, V, layer, s, e, q, scale, last, gen):
    B, H, S = K.shape[1], K.shape[2], K.shape[4]
    m0 = torch.rand(B, H, S, generator=gen, device="cuda") * (2.0 if last % 2 else 0.0)
    want, tol, mass, mtol = W.attend_ref(K[layer], V[layer], s, e, q, scale, last=last, mass=m0)
    for b, _, a, z in R.spans(s, e):  # nothing past a sequence's rows is attended
        K[:, b, :, :, z:] = math.nan
        V[:, b, :, z:] = math.nan
        m0[b, :, z:] = math.nan
    got_mass = m0.clone()
    got = _attend(cache, layer, s, e, q, scale, got_mass, last)
    R.assert_within(got, want, tol, "outputs")
    for b, _, a, z in R.spans(s, e):
        z = z if z > a else 0
        R.assert_within(got_mass[b, :, :z], mass[b, :, :z], mtol[b, :, :z], "weights")
        assert torch.equal(got_mass[b, :, z:].view(torch.int32), m0[b, :, z:].view(torch.int32))
    again = m0.clone()  # the same bits again
    assert torch.equal(_attend(cache, layer, s, e, q, scale, again, last).view(torch.int16), got.view(torch.int16))
    assert torch.equal(again.view(torch.int32), got_mass.view(torch.int32))


CASES = [
    # B, H, G, D, S, ctx, new, last
    (1, 1, 1, 64, 1, (0, 0), (1, 1), 0),
    (2, 2, 1, 64, 300, (0, 299), (1, 1), 0),
    (3, 2, 1, 128, 700, (100, 690), (1, 1), 1),
    (3, 2, 4, 128, 1024, (0, 1000), (1, 4), 0),       # scores kept
    (3, 2, 4, 128, 1024, (0, 1000), (1, 9), 3),       # one row tile, scores not kept
    (2, 2, 8, 64, 2000, (900, 1900), (1, 2), 1),
    (2, 1, 71, 64, 400, (0, 390), (1, 3), 0),
    (1, 1, 128, 128, 500, (400, 440), (33, 33), 5),
    (2, 3, 1, 64, 1300, (0, 100), (600, 1200), 0),
    (2, 2, 1, 128, 1500, (0, 0), (1, 1500), 64),
    (3, 2, 3, 64, 421, (0, 100), (0, 321), 0),
    (2, 2, 2, 8, 1024, (512, 600), (300, 400), 32),
    (2, 2, 1, 72, 517, (0, 129), (250, 388), 0),       # an odd S: rows of one chunk a run
    (2, 1, 5, 96, 1261, (900, 900), (200, 255), 0),
    (2, 1, 2, 120, 2000, (1500, 1700), (255, 256), 1000),
    (36, 2, 1, 64, 200, (0, 120), (0, 60), 7),
    (40, 2, 4, 64, 100, (0, 90), (0, 2), 0),
    (1, 2, 1, 128, 4096, (2048, 2048), (2048, 2048), 0),
    (1, 1, 2, 64, 20000, (19500, 19500), (300, 300), 64),
    (1, 2, 4, 128, 30000, (29000, 29900), (1, 1), 0),  # cut among many CTAs
    (1, 1, 1, 64, 9000, (0, 0), (9000, 9000), 0),
    (4, 64, 1, 128, 1500, (600, 900), (40, 600), 0),    # more units than SMs
    (5, 70, 1, 128, 1200, (0, 1130), (1, 16), 9),
    (2, 3, 16, 64, 900, (300, 400), (1, 1), 0),
    # many units of few rows: two heads at a time, an odd number of them, cut among CTAs
    (11, 71, 1, 128, 700, (0, 690), (1, 3), 2),
    (10, 63, 4, 64, 500, (300, 480), (0, 16), 0),
    (310, 2, 2, 40, 321, (0, 300), (1, 5), 3),
    (3, 301, 1, 72, 900, (800, 899), (1, 1), 0),
    (10, 61, 16, 64, 300, (200, 299), (1, 1), 0),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B, H, G, D, S, ctx, new, last", CASES)
def test_scored_attention(dtype, B, H, G, D, S, ctx, new, last):
    rng = np.random.default_rng(S + last)
    gen = _gen(S + D)
    s = rng.integers(ctx[0], ctx[1] + 1, size=B).astype(np.int32)
    n = rng.integers(new[0], new[1] + 1, size=B).astype(np.int32)
    if new[0] == 0 and B > 1:
        n[rng.integers(B)] = 0
    e = (s + np.minimum(n, S - s)).astype(np.int32)
    cache, K, V = R.make_cache(dtype, 2, B, H, D, S, gen)
    q = torch.empty(int((e - s).sum()), H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) * 2
    _check(cache, K, V, 1, s, e, q, D ** -0.5, last, gen)


@pytest.mark.parametrize("seed", range(24))
def test_random_scored_attention(seed):
    rng = np.random.default_rng(seed)
    gen = _gen(seed)
    dtype = ["fp16", "bf16"][rng.integers(2)]
    B, H, G, D = int(rng.integers(1, 9)), int(rng.integers(1, 9)), int(rng.integers(1, 9)), 8 * int(rng.integers(1, 17))
    s = rng.integers(0, int(rng.choice([1, 200, 3000])), size=B).astype(np.int32)
    e = s + rng.integers(0, int(rng.choice([2, 5, 60, 700])), size=B).astype(np.int32)
    S = int(e.max()) + int(rng.integers(0, 9)) + 1
    cache, K, V = R.make_cache(dtype, 1, B, H, D, S, gen)
    wide = torch.empty(int((e - s).sum()), H * G * D + 24, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    q = wide[:, 8:8 + H * G * D].view(-1, H * G, D)  # strided tokens
    _check(cache, K, V, 0, s, e, q, 0.2, int(rng.choice([0, 0, 1, 5, 64])), gen)


def test_outputs_are_those_of_prompt_attention():
    gen = _gen(5)
    s, e = np.array([0, 40, 300], np.int32), np.array([200, 41, 500], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 3, 2, 64, 512, gen)
    q = torch.empty(401, 4, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    want = torch.empty_like(q)
    dv.dv_prompt_attention(cache, 0, s, e, q, want, 0.125, _ws(cache, s, e, 4))
    mass = torch.zeros(3, 2, 512, device="cuda")
    assert torch.equal(_attend(cache, 0, s, e, q, 0.125, mass), want)
    # every token's weights sum to one for each of its query heads (the bound of a weight in
    # bounded_refs.weights_ref is below 2^-13 here, for at most 400 of them)
    total = mass.double().sum(-1)
    assert float((total - torch.tensor([400., 2., 400.], device="cuda")[:, None]).abs().max()) < 400 * 2.0 ** -13


@pytest.mark.parametrize("new, last", [(1, 0), (4, 0), (4, 2), (200, 0), (200, 50)])
def test_weights_that_are_not_numbers_stay_with_the_rows_attended(new, last):
    """A query of NaN, and one whose scores are all -inf, make the rows that they attend NaN where
    they are counted; later rows, other heads and other sequences keep their numbers."""
    gen = _gen(21)
    s, e = np.array([300, 290], np.int32), np.array([300 + new, 290 + new], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 2, 2, 64, 512, gen)
    q = torch.empty(2 * new, 4, 64, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    at = 0 if new < 5 else 60
    q[at, 1] = math.nan            # sequence 0, key head 0
    K[0, 1, 1] = 0                 # sequence 1, key head 1
    K[0, 1, 1, 0, :, 0] = 1.0
    q[new + at, 2, 0] = -math.inf  # every score -inf ...
    q[new + at, 2, 1:] = 0.0       # (and no infinity times zero)
    K[0, 1, 1, :, :, 1:] = 0.0
    mass = torch.zeros(2, 2, 512, device="cuda")
    _attend(cache, 0, s, e, q, 0.125, mass, last)
    counted = last == 0 or at >= new - last
    want = torch.zeros(2, 2, 512, dtype=torch.bool, device="cuda")
    want[0, 0, :300 + at + 1] = want[1, 1, :290 + at + 1] = counted
    assert torch.equal(mass.isnan(), want)
    plain = torch.zeros_like(mass)  # what is a number is what it is without those queries' heads
    q2 = torch.nan_to_num(q, nan=0.0, posinf=0.0, neginf=0.0)
    _attend(cache, 0, s, e, q2, 0.125, plain, last)
    clean = ~want
    clean[0, 0] = clean[1, 1] = False
    assert torch.equal(mass[clean], plain[clean])


def test_scored_in_a_graph_on_a_side_stream():
    gen = _gen(11)
    for e in ([701, 300], [701, 1]):  # with a prompt; decode steps, whose scores are kept
        s, e = np.array([700, 0], np.int32), np.array(e, np.int32)
        cache, K, V = R.make_cache("bf16", 1, 2, 4, 128, 1024, gen)
        q = torch.empty(int((e - s).sum()), 8, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        out, ws, mass = torch.zeros_like(q), _ws(cache, s, e, 8), torch.zeros(2, 4, 1024, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            dv.dv_scored_attention(cache, 0, s, e, q, out, 0.1, mass, ws, stream=side)
        for _ in range(3):
            q.normal_(generator=gen)
            K.normal_(generator=gen)
            before = mass.clone()
            graph.replay()
            torch.cuda.synchronize()
            want, tol, m, mtol = W.attend_ref(K[0], V[0], s, e, q, 0.1, mass=before)
            R.assert_within(out, want, tol)
            R.assert_within(mass, m, mtol)


def test_two_streams_in_flight_together():
    """Prompts on one stream, decode steps of another cache on a second, several calls each:
    the bits of the same calls one after the other."""
    gen = _gen(31)
    jobs = []
    for s, e, H, G in (([0, 10, 300], [900, 500, 800], 6, 2), ([700, 20, 900], [701, 21, 901], 24, 4)):
        s, e = np.array(s, np.int32), np.array(e, np.int32)
        cache, K, V = R.make_cache("bf16", 1, 3, H, 128, 1024, gen)
        q = torch.empty(int((e - s).sum()), H * G, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        jobs.append((cache, s, e, q, torch.zeros_like(q), _ws(cache, s, e, H * G), torch.zeros(3, H, 1024, device="cuda"),
                     torch.cuda.Stream()))
    def call(j, stream):
        cache, s, e, q, out, ws, mass, _ = j
        for _ in range(5):
            dv.dv_scored_attention(cache, 0, s, e, q, out, 0.1, mass, ws, last=100, stream=stream)
    want = []
    for j in jobs:
        call(j, None)
        torch.cuda.synchronize()
        want.append((j[4].clone(), j[6].clone()))
        j[4].zero_()
        j[6].zero_()
    torch.cuda.synchronize()
    for j in jobs:
        call(j, j[-1])
    torch.cuda.synchronize()
    for j, (out, mass) in zip(jobs, want):
        assert torch.equal(j[4], out) and torch.equal(j[6], mass)


@pytest.mark.parametrize("new", [1, 700])
def test_a_wait_that_gives_up_is_reported(new):
    gen = _gen(12)
    s, e = np.array([700 - new], np.int32), np.array([700], np.int32)
    cache, K, V = R.make_cache("fp16", 1, 1, 2, 64, 700, gen)
    q = torch.empty(new, 2, 64, dtype=torch.float16, device="cuda").normal_(generator=gen)
    mass = torch.zeros(1, 2, 700, device="cuda")
    dv.dv_attention_check()
    for tries in (0, 1, 3):
        dv.dv_debug_attention_tries(tries)
        try:
            _attend(cache, 0, s, e, q, 0.125, mass)
            torch.cuda.synchronize()
        finally:
            dv.dv_debug_attention_tries()
        if tries == 0:
            with pytest.raises(dv.DvError) as ei:
                dv.dv_attention_check()
            assert ei.value.status == dv.DV_ERR_TIMEOUT
    try:
        dv.dv_attention_check()
    except dv.DvError as x:
        assert x.status == dv.DV_ERR_TIMEOUT
    _check(cache, K, V, 0, s, e, q, 0.125, 0, gen)

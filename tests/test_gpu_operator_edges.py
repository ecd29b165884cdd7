"""The operators over the cache at their edges: streams other than torch's current
one, values at the ends of their types, and offsets past what 32 bits hold."""
import math

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv
from tests import operator_refs as R

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _stream_of(t):
    """The stream whose order torch reuses the tensor's memory in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


@pytest.mark.parametrize("handle", [False, True], ids=["object", "handle"])
def test_rotated_queries_are_allocated_under_the_stream_that_writes_them(handle):
    gen = _gen(31)
    s, e = np.array([3, 0], np.int32), np.array([300, 200], np.int32)
    T, H, D = 497, 4, 64
    cache, K, V = R.make_cache("bf16", 1, 2, H, D, 320, gen)
    q, k, v = (torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(3))
    rope = dv.Rope(D)
    want = dv.dv_kv_append(cache, 0, s, e, k, v, q=q, rope=rope)
    assert _stream_of(want) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    gone = torch.empty_like(q)  # a block that the current stream's pool can hand out again
    ptr = gone.data_ptr()
    torch.cuda.synchronize()
    del gone
    got = dv.dv_kv_append(cache, 0, s, e, k, v, q=q, rope=rope, stream=side.cuda_stream if handle else side)
    assert got.data_ptr() != ptr and _stream_of(got) == side.cuda_stream
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):  # the current stream, named or not
        assert _stream_of(dv.dv_kv_append(cache, 0, s, e, k, v, q=q, rope=rope)) == side.cuda_stream
        other = dv.dv_kv_append(cache, 0, s, e, k, v, q=q, rope=rope, stream=0)
        assert _stream_of(other) == torch.cuda.default_stream().cuda_stream
    torch.cuda.synchronize()
    assert torch.equal(other, want)


# ---- scores and values at the ends of their types --------------------------------------

def _attend(cache, s, e, q, scale, tree=None, prompt=False):
    n = dv.dv_attention_workspace(cache, s, e, q.shape[1])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    out = torch.full_like(q, 7.0)
    if prompt:
        dv.dv_prompt_attention(cache, 0, s, e, q, out, scale, ws)
    else:
        dv.dv_tree_attention(cache, 0, s, e, q, out, scale, ws, tree=tree)
    return out


# one tile, tiles of both chains, pieces joined through the workspace
LENGTHS = [(0, 3), (100, 5), (300, 20), (20000, 2), (9000, 33), (5, 700), (6000, 150)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("ctx, n", LENGTHS)
def test_a_query_of_nan_gives_nan_however_its_rows_are_divided(dtype, ctx, n):
    H, G, D = 2, 4, 64
    gen = _gen(ctx + n)
    s, e = np.array([ctx], np.int32), np.array([ctx + n], np.int32)
    cache, K, V = R.make_cache(dtype, 1, 1, H, D, ctx + n, gen)
    q = torch.empty(n, H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 0.125)
    q[n - 1, 3, 5] = math.nan
    want[n - 1, 3] = math.nan
    for prompt in (False, True):
        if prompt or n <= 64:
            R.assert_within(_attend(cache, s, e, q, 0.125, prompt=prompt), want, tol)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("ctx, n", LENGTHS)
@pytest.mark.parametrize("part", [1.0, 0.6])
def test_scores_of_minus_infinity(dtype, ctx, n, part):
    """Rows whose score is -inf have no weight; where every attended row is one,
    the softmax is 0 / 0.  (A token that attends no row at all has zeros.)"""
    H, G, D = 2, 4, 64
    gen = _gen(ctx + n + 1)
    s, e = np.array([ctx], np.int32), np.array([ctx + n], np.int32)
    cache, K, V = R.make_cache(dtype, 1, 1, H, D, ctx + n, gen)
    K[0, 0, 0, 0, :int(part * (ctx + n)), 0] = -math.inf  # element 0 of key head 0
    q = torch.empty(n, H * G, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    q[:, :, 0] = 1.0
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 0.125)
    last = torch.arange(ctx, ctx + n, device="cuda")  # the last row that each token attends
    want[last < int(part * (ctx + n)), :G] = math.nan
    for prompt in (False, True):
        if prompt or n <= 64:
            R.assert_within(_attend(cache, s, e, q, 0.125, prompt=prompt), want, tol)


def test_masks_of_rows_of_minus_infinity_and_masks_of_nothing():
    H, D, n = 2, 64, 4
    gen = _gen(3)
    s, e = np.array([0], np.int32), np.array([n], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 1, H, D, n, gen)
    K[0, 0, 0, 0, 1, 0] = -math.inf
    q = torch.ones(n, H, D, dtype=torch.bfloat16, device="cuda")
    bits = [0b0001, 0b0010, 0b0000, 0b0110]
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 0.125, bits)
    want[1, 0] = math.nan
    got = _attend(cache, s, e, q, 0.125, tree=R.bits_tensor(bits))
    R.assert_within(got, want, tol)
    assert not got[2].any()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("row", [5, 130, 260])
def test_values_of_nan_reach_tokens_that_give_them_no_weight(dtype, row):
    """0 x NaN is NaN in whichever chain of tiles the row lies."""
    H, D, ctx = 2, 64, 300
    gen = _gen(row)
    s, e = np.array([ctx], np.int32), np.array([ctx + 1], np.int32)
    cache, K, V = R.make_cache(dtype, 1, 1, H, D, ctx + 1, gen)
    lo = row // 128 * 128
    K[0, 0, :, 0, lo:lo + 128, 0] = -400.0
    V[0, 0, 0, row, 3] = math.nan
    q = torch.empty(1, H, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen)
    q[:, :, 0] = 40.0  # scores of -2000 beside ordinary ones
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 0.125)
    assert torch.isnan(want[0, 0, 3]) and torch.isfinite(want[0, 1]).all()
    R.assert_within(_attend(cache, s, e, q, 0.125), want, tol)


@pytest.mark.parametrize("peak", [0, 70000, 131071])
@pytest.mark.parametrize("nats", [9.0, 17.0])
@pytest.mark.parametrize("n", [1, 200])
def test_the_many_small_weights_below_a_peak(peak, nats, n):
    """fp16: 131071 keys far below one peak have a good part of the output between
    them. attention_ref's bound allows each weight 2^-25 of the largest; they
    are held to 2^-32 (half a step of fp16's smallest, 2^-25, of weights 2^7 times
    as large)."""
    H, D, S = 1, 64, 131072 + n
    gen = _gen(peak + n)
    s, e = np.array([131072], np.int32), np.array([S], np.int32)
    cache, K, V = R.make_cache("fp16", 1, 1, H, D, S, gen, fill=0.0)
    V[0, 0, 0] = torch.rand(S, D, device="cuda", generator=gen).to(torch.float16)
    K[0, 0, 0, 0, peak, 0], V[0, 0, 0, peak] = nats, 0.0
    q = torch.zeros(n, H, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 1.0)
    tol -= (2.0 ** -25 - 2.0 ** -32) * V[0, 0, 0].double().abs().sum(0)
    if n <= 64:
        R.assert_within(_attend(cache, s, e, q, 1.0), want, tol)
    R.assert_within(_attend(cache, s, e, q, 1.0, prompt=True), want, tol)


@pytest.mark.parametrize("peak", [0, 9000])
@pytest.mark.parametrize("n", [1, 200])
def test_the_many_small_weights_of_undivided_rows(peak, n):
    """As above with two heads for each SM, so that no head's rows are divided: the
    peak is the reference of all of its row's weights."""
    H, D, ctx = 2 * torch.cuda.get_device_properties(0).multi_processor_count, 64, 16384
    gen = _gen(peak + n)
    s, e = np.array([ctx], np.int32), np.array([ctx + n], np.int32)
    cache, K, V = R.make_cache("fp16", 1, 1, H, D, ctx + n, gen, fill=0.0)
    V[0, 0] = torch.rand(H, ctx + n, D, device="cuda", generator=gen).to(torch.float16)
    K[0, 0, :, 0, peak, 0], V[0, 0, :, peak] = 17.0, 0.0
    q = torch.zeros(n, H, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 1.0)
    tol -= (2.0 ** -25 - 2.0 ** -32) * V[0, 0].double().abs().sum(1)
    for prompt in (False, True):
        if prompt or n <= 64:
            R.assert_within(_attend(cache, s, e, q, 1.0, prompt=prompt), want, tol)


# ---- waits that give up ------------------------------------------------------------------

def _gives_up(stream=None):
    """Whether the check reports a wait that gave up."""
    try:
        dv.dv_attention_check(stream)
        return False
    except dv.DvError as err:
        assert err.status == dv.DV_ERR_TIMEOUT
        return True


@pytest.fixture
def few_tries():
    dv.dv_attention_check()
    yield dv.dv_debug_attention_tries
    dv.dv_debug_attention_tries(-1)
    torch.cuda.synchronize()
    _gives_up()  # (a record that a failed test has left)


@pytest.mark.parametrize("H, G, D, ctx, n", [
    (1, 1, 64, 0, 1),        # one unit of one tile: everything is loaded without a wait
    (2, 4, 64, 300, 5),
    (2, 4, 128, 5000, 40),   # rings that fill, pieces that are joined
    (200, 1, 128, 700, 9),   # more units than SMs
    (3, 1, 72, 100, 600),
    (40, 2, 128, 0, 700),
])
def test_a_wait_that_gives_up_ends_in_a_status(few_tries, H, G, D, ctx, n):
    """With no tries at all every wait gives up at once, with copies in flight and
    tensor memory held; with a few, here and there. The kernel ends, the check
    says so once, and the next call works."""
    gen = _gen(ctx + n)
    s, e = np.array([ctx, 0], np.int32), np.array([ctx + n, 1], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 2, H, D, ctx + n, gen)
    q = torch.empty(n + 1, H * G, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 0.125)
    for prompt in (False, True):
        if n > 64 and not prompt:
            continue
        for tries in (0, 1, 2, 3, 5, 10, 30, 100):
            few_tries(tries)
            for _ in range(3):
                _attend(cache, s, e, q, 0.125, prompt=prompt)
            assert _gives_up() or tries > 0
            assert not _gives_up()
            few_tries(-1)
            R.assert_within(_attend(cache, s, e, q, 0.125, prompt=prompt), want, tol)
            assert not _gives_up()


def test_every_streams_check_reports_a_wait_that_gave_up(few_tries):
    """One caller's check takes no other caller's record away."""
    s, e = np.array([300], np.int32), np.array([305], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 1, 2, 64, 305, _gen(1))
    q = torch.ones(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        _gives_up(st)
        assert not _gives_up(st)
    torch.cuda.synchronize()
    few_tries(0)
    for st in streams:
        with torch.cuda.stream(st):
            _attend(cache, s, e, q, 0.125)
    few_tries(-1)
    torch.cuda.synchronize()
    for st in streams:
        assert _gives_up(st)
    for st in streams:
        assert not _gives_up(st)
    assert _gives_up() and not _gives_up()  # the current stream's, which has seen none of it
    with torch.cuda.stream(streams[0]):
        _attend(cache, s, e, q, 0.125)
    assert not any(_gives_up(st) for st in streams)


def test_the_check_is_refused_in_a_capture_and_leaves_it_whole():
    s, e = np.array([300], np.int32), np.array([305], np.int32)
    cache, K, V = R.make_cache("bf16", 1, 1, 2, 64, 305, _gen(2))
    q = torch.ones(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    want = _attend(cache, s, e, q, 0.125)
    out = torch.zeros_like(q)
    n = dv.dv_attention_workspace(cache, s, e, 2)
    ws = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    dv.dv_attention_check()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        dv.dv_tree_attention(cache, 0, s, e, q, out, 0.125, ws)
        with pytest.raises(dv.DvError) as ei:
            dv.dv_attention_check(side)
        assert ei.value.status == dv.DV_ERR_INVALID_ARG
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    dv.dv_attention_check()


# ---- offsets past 32 bits ----------------------------------------------------------------

def test_chunk_offsets_past_32_bits():
    """One layer of more than 2^31 16-byte chunks: the last heads' rows lie past
    what a 32-bit chunk index reaches, in full tiles and in a partial one, with
    values of their own in every head and a non-finite one among the last's."""
    H, G, D, S, ctx, n = 131, 2, 128, (1 << 20) + 37, 295, 6
    need = H * D * S * 2
    if torch.cuda.mem_get_info()[0] < 2 * need + (8 << 30):
        pytest.skip("needs 80 GB of free device memory")
    assert (H - 1) * (D // 8) * S > 1 << 31
    gen = _gen(8)
    k, v = (torch.empty(H * D * S, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = dv.Cache(1, 1, H, D, S, 2, k, v)
    K, V = k.view(1, 1, H, D // 8, S, 8), v.view(1, 1, H, S, D)
    end = ctx + n
    K[0, 0, :, :, :end + 9].normal_(generator=gen)
    V[0, 0, :, :end + 9].normal_(generator=gen)
    K[0, 0, :, :, S - 9:], V[0, 0, :, S - 9:] = 3.0, 4.0
    new = torch.empty(n, (G + 2) * H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    s, e = np.array([ctx], np.int32), np.array([end], np.int32)
    before = K[0, 0, :, :, :end + 9].clone(), V[0, 0, :, :end + 9].clone()
    new[2, (G + 2) * H - 1, 7] = math.inf  # the last head's value of the third new token

    # append, at the context's end and at the cache's
    q = dv.dv_kv_append(cache, 0, s, e, new[:, G * H:(G + 1) * H], new[:, (G + 1) * H:], q=new[:, :G * H])
    assert torch.equal(q, new[:, :G * H])
    dv.dv_kv_append(cache, 0, np.array([S - n], np.int32), np.array([S], np.int32), new[:, G * H:(G + 1) * H],
                    new[:, (G + 1) * H:])
    for at in (ctx, S - n):
        assert torch.equal(K[0, 0, :, :, at:at + n].permute(2, 0, 1, 3).reshape(n, H, D), new[:, G * H:(G + 1) * H])
        assert torch.equal(V[0, 0, :, at:at + n].transpose(0, 1), new[:, (G + 1) * H:])
    for now, was, dim in ((K[0, 0], before[0], 2), (V[0, 0], before[1], 1)):
        assert torch.equal(now.narrow(dim, 0, ctx), was.narrow(dim, 0, ctx))
        assert torch.equal(now.narrow(dim, end, 9), was.narrow(dim, end, 9))
    assert (K[0, 0, :, :, S - 9:S - n] == 3).all() and (V[0, 0, :, S - 9:S - n] == 4).all()

    # attention: two full tiles and a partial one of every head
    want, tol = R.attention_ref(K[0], V[0], s, e, q, D ** -0.5)
    assert torch.isinf(want[2:, (H - 1) * G:, 7]).all() and torch.isfinite(want[:2]).all()
    R.assert_within(_attend(cache, s, e, q, D ** -0.5), want, tol)
    R.assert_within(_attend(cache, s, e, q, D ** -0.5, prompt=True), want, tol)

    # compact, at both ends
    for at in (ctx, S - n):
        rows = K[0, 0, :, :, at:at + n].clone(), V[0, 0, :, at:at + n].clone()
        keep = torch.tensor([at + 1, at + 3, at + 5], dtype=torch.int32, device="cuda")
        dv.dv_kv_compact(cache, 0, 1, np.array([at], np.int32), np.array([at + 3], np.int32), keep)
        assert torch.equal(K[0, 0, :, :, at:at + 3], rows[0][:, :, [1, 3, 5]])
        assert torch.equal(V[0, 0, :, at:at + 3], rows[1][:, [1, 3, 5]])
        assert torch.equal(K[0, 0, :, :, at + 3:at + n], rows[0][:, :, 3:])
        assert torch.equal(V[0, 0, :, at + 3:at + n], rows[1][:, 3:])
    del k, v, K, V, cache
    torch.cuda.empty_cache()

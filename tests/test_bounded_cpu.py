"""What the operators that keep a cache within a bound refuse, before any pointer is
used (CPU)."""
import math

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv

F16 = torch.float16
S2, E2 = np.array([4, 0], np.int32), np.array([6, 3], np.int32)  # 5 new tokens


def _cache(L=2, B=2, H=4, D=64, S=32, P=2):
    return dv.Cache(L, B, H, D, S, P, 0x1000, 0x2000)  # never dereferenced


def _refused(status, fn):
    with pytest.raises(dv.DvError) as ei:
        fn()
    assert ei.value.status == status, ei.value
    return str(ei.value)


def _qo(n=5, heads=8, D=64, dt=F16):
    return torch.zeros(n, heads, D, dtype=dt), torch.zeros(n, heads, D, dtype=dt)


def test_window_refusals():
    def call(c=None, layer=0, s=S2, e=E2, q=None, scale=0.125, heads=8, D=64, window=4, sinks=1):
        q, o = _qo(int((np.asarray(e) - np.asarray(s)).sum()), heads, D) if q is None else q
        dv.dv_window_attention(c or _cache(), layer, s, e, q, o, scale, window, sinks, None, stream=0)

    for window, sinks in ((0, 0), (-1, 0), (-2**31, 0), (1, -1), (4, -2**31)):
        _refused(dv.DV_ERR_INVALID_ARG, lambda: call(window=window, sinks=sinks))
    for kw in (dict(window=2**31), dict(window=2**32 + 4), dict(sinks=2**31), dict(sinks=-2**31 - 1)):
        with pytest.raises(ValueError):
            call(**kw)
    _refused(dv.DV_ERR_RANGE, lambda: call(layer=2))
    _refused(dv.DV_ERR_RANGE, lambda: call(layer=-1))
    _refused(dv.DV_ERR_RANGE, lambda: call(s=[4, 0], e=[33, 0]))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(heads=6))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(heads=4 * 129))
    for scale in (0.0, -1.0, math.inf, math.nan):
        _refused(dv.DV_ERR_INVALID_ARG, lambda: call(scale=scale))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(D=136), D=136))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(P=4)))
    with pytest.raises(TypeError):
        call(q=_qo(dt=torch.float32))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(q=_qo(n=4)))
    with pytest.raises(ValueError):
        call(q=(_qo()[0], _qo(n=4)[1]))
    call(s=[4, 3], e=[4, 3])  # nothing to do: no pointer is looked at
    n = np.zeros(2, np.int32).ctypes.data
    assert dv.lib.dv_window_attention(None, 0, n, n, None, 4, 1, None, None, 0, None) == dv.DV_ERR_INVALID_ARG
    assert dv.lib.dv_window_attention(_cache().ref, 0, n, n, None, 4, 1, None, None, 0, None) == dv.DV_ERR_INVALID_ARG


def test_window_refusals_of_trees():
    def call(n=5, window=64, bits=None, c=None, s=S2, e=E2):
        q, o = _qo(n)
        bits = torch.ones(n, dtype=torch.int64) if bits is None else bits
        dv.dv_window_attention(c or _cache(), 0, s, e, q, o, 0.125, window, 1, None, tree=bits, stream=0)

    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(window=63))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(n=65, c=_cache(S=200), s=[4, 0], e=[69, 0]))
    for bits in (torch.ones(4, dtype=torch.int64), torch.ones(5, dtype=torch.int32)):
        with pytest.raises(ValueError):
            call(bits=bits)


def test_scored_refusals():
    def call(c=None, layer=0, s=S2, e=E2, q=None, scale=0.125, heads=8, D=64, last=0, mass=None):
        c = c or _cache()
        q, o = _qo(int((np.asarray(e) - np.asarray(s)).sum()), heads, D) if q is None else q
        mass = torch.zeros(2, 4, 32) if mass is None else mass
        dv.dv_scored_attention(c, layer, s, e, q, o, scale, mass, None, last=last, stream=0)

    for last in (-1, -2**31):
        _refused(dv.DV_ERR_INVALID_ARG, lambda: call(last=last))
    with pytest.raises(ValueError):
        call(last=2**31)
    for mass in (torch.zeros(2, 4, 31), torch.zeros(4, 32), torch.zeros(2, 2, 4, 32)):
        with pytest.raises(ValueError):
            call(mass=mass)
    for mass in (torch.zeros(2, 4, 32, dtype=torch.float64), torch.zeros(2, 4, 32, dtype=F16),
                 torch.zeros(2, 4, 32, dtype=torch.int32), torch.zeros(2, 4, 64)[..., ::2]):
        with pytest.raises(TypeError):
            call(mass=mass)
    _refused(dv.DV_ERR_RANGE, lambda: call(layer=2))
    _refused(dv.DV_ERR_RANGE, lambda: call(s=[4, 0], e=[33, 0]))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(heads=6))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(scale=math.nan))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(D=136), D=136))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(P=4)))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(q=_qo(n=4)))
    _refused(dv.DV_ERR_BUFFER_TOO_SMALL, lambda: call())  # no workspace
    call(s=[4, 3], e=[4, 3])
    n = np.zeros(2, np.int32).ctypes.data
    assert dv.lib.dv_scored_attention(None, 0, n, n, None, 0, None, None, 0, None) == dv.DV_ERR_INVALID_ARG


def test_scored_refuses_weights_on_other_buffers():
    K, V = (torch.zeros(2, 4 * 64 * 32, dtype=F16) for _ in range(2))
    c = dv.Cache(2, 1, 4, 64, 32, 2, K, V)
    s, e = np.array([4], np.int32), np.array([9], np.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    q, o = _qo(n=64, heads=4)
    mass = torch.zeros(4 * 32)

    def call(**kw):
        a = dict(q=q[:5], out=o[:5], mass=mass, ws=ws) | kw
        dv.dv_scored_attention(c, 1, s, e, a["q"], a["out"], 0.1, a["mass"].view(1, 4, 32), a["ws"], stream=0)

    for kw in (dict(mass=K[1].view(torch.float32)[40:168]), dict(mass=V[1].view(torch.float32)[-128:]),
               dict(mass=q.view(-1).view(torch.float32)[600:728]), dict(mass=o.view(-1).view(torch.float32)[:128]),
               dict(mass=ws.view(torch.float32)[64:192])):
        _refused(dv.DV_ERR_INVALID_ARG, lambda: call(**kw))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(out=q[4:9]))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(ws=(K.data_ptr(), 1 << 20)))


def test_scored_workspace_refusals():
    assert dv.dv_scored_attention_workspace(_cache(), S2, E2, 8) >= dv.dv_attention_workspace(_cache(), S2, E2, 8)
    assert dv.dv_scored_attention_workspace(_cache(), [3, 3], [3, 3], 8) == 0
    _refused(dv.DV_ERR_INVALID_ARG, lambda: dv.dv_scored_attention_workspace(_cache(), S2, E2, 6))
    _refused(dv.DV_ERR_RANGE, lambda: dv.dv_scored_attention_workspace(_cache(), [0, 0], [33, 0], 8))


def test_evict_refusals():
    def call(c=None, l0=0, l1=2, rows=(20, 32), kept=(10, 32), sinks=1, recent=2, mass=None, keep=None, out=None):
        c = c or _cache()
        mass = torch.zeros(max(0, l1 - l0), 2, 4, 32) if mass is None else mass
        keep = torch.zeros(max(0, l1 - l0) * 4 * int(np.sum(kept)), dtype=torch.int32) if keep is None else keep
        dv.dv_kv_evict(c, l0, l1, rows, kept, sinks, recent, mass, keep, mass_out=out, stream=0)

    _refused(dv.DV_ERR_RANGE, lambda: call(l1=3))
    _refused(dv.DV_ERR_RANGE, lambda: call(l0=-1, l1=1))
    _refused(dv.DV_ERR_RANGE, lambda: call(rows=(20, 33), kept=(10, 10)))
    _refused(dv.DV_ERR_RANGE, lambda: call(rows=(20, 9), kept=(10, 10)))
    _refused(dv.DV_ERR_RANGE, lambda: call(kept=(-1, 10), keep=torch.zeros(72, dtype=torch.int32)))
    for sinks, recent in ((-1, 0), (0, -1), (6, 5), (11, 0), (0, 11), (2**31 - 1, 2**31 - 1)):
        _refused(dv.DV_ERR_INVALID_ARG, lambda: call(sinks=sinks, recent=recent))
    for kw in (dict(sinks=2**31), dict(recent=2**32 + 1)):
        with pytest.raises(ValueError):
            call(**kw)
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(keep=torch.zeros(335, dtype=torch.int32)))
    for bad in (torch.zeros(2, 2, 4, 31), torch.zeros(1, 2, 4, 32)):
        with pytest.raises(ValueError):
            call(mass=bad)
        with pytest.raises(ValueError):
            call(out=bad)
    with pytest.raises(TypeError):
        call(mass=torch.zeros(2, 2, 4, 32, dtype=torch.int32))
    with pytest.raises(ValueError):
        call(keep=torch.zeros(336, dtype=torch.int64))
    buf = torch.zeros(2 * 2 * 4 * 32 + 8)
    a, b = buf[:512].view(2, 2, 4, 32), buf[4:516].view(2, 2, 4, 32)
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(mass=a, out=b))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(mass=a, keep=buf.view(torch.int32)[100:436]))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(out=a, keep=buf.view(torch.int32)[100:436]))
    K, V = (torch.zeros(2, 2 * 4 * 64 * 32, dtype=F16) for _ in range(2))
    c = dv.Cache(2, 2, 4, 64, 32, 2, K, V)
    on = V[1].view(torch.float32)[16:272].view(1, 2, 4, 32)
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(c=c, l0=1, mass=on))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(c=c, l0=1, out=on))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(c=c, l0=1, keep=K[1].view(torch.int32)[:168]))
    call(l0=1, l1=1)
    call(rows=(0, 0), kept=(0, 0))
    n = np.zeros(2, np.int32).ctypes.data
    assert dv.lib.dv_kv_evict(None, 0, 1, n, n, 0, 0, None, None, None, 0, None) == dv.DV_ERR_INVALID_ARG
    assert dv.lib.dv_kv_evict(_cache().ref, 0, 1, None, n, 0, 0, None, None, None, 0, None) == dv.DV_ERR_INVALID_ARG


def test_rows_that_32_bits_hardly_count_are_refused():
    S = 2**31 - 16384
    c = dv.Cache(1, 1, 1, 8, S, 2, 0x1000, 0x2000)
    q, o = _qo(n=1, heads=1, D=8)
    n = np.zeros(1, np.int32).ctypes.data
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: dv.dv_window_attention(c, 0, [S - 1], [S], q, o, 0.1, 4, 1, None, stream=0))
    a = dv.dv.dv_queries(dv.DV_DTYPE_FP16, 1, 0, None, 8, None, 8, 0.1)
    import ctypes
    assert dv.lib.dv_scored_attention(c.ref, 0, n, n, ctypes.byref(a), 0, None, None, 0, None) == dv.DV_ERR_UNSUPPORTED
    assert dv.lib.dv_kv_evict(c.ref, 0, 1, n, n, 0, 0, None, None, None, 0, None) == dv.DV_ERR_UNSUPPORTED


@pytest.mark.parametrize("seed", range(8))
def test_the_workspace_of_causal_attention_is_enough_for_any_window(seed):
    """The size check comes before any pointer is looked up: what is refused here is not the size."""
    rng = np.random.default_rng(seed)
    for _ in range(60):
        B, H, G = int(rng.integers(1, 40)), int(rng.integers(1, 90)), int(rng.choice([1, 2, 3, 4, 8, 71, 128]))
        S = int(np.exp(rng.uniform(1, 9)))
        s = rng.integers(0, S, size=B).astype(np.int32)
        e = np.minimum(S, s + rng.integers(0, int(rng.choice([2, 4, 70, 700])), size=B)).astype(np.int32)
        n = int((e - s).sum())
        if n * H * G > 1 << 21:  # (some megabytes of tokens)
            continue
        c = dv.Cache(1, B, H, 64, S, 2, 0x1000, 0x2000)
        q, o = torch.empty(n, H * G, 64, dtype=F16), torch.empty(n, H * G, 64, dtype=F16)
        size = dv.dv_attention_workspace(c, s, e, H * G)
        for window, sinks in ((1, 0), (1, 1), (5, 33), (100, 4), (129, 128), (S, 0)):
            try:
                dv.dv_window_attention(c, 0, s, e, q, o, 0.1, window, sinks, (1 << 40, size), stream=0)
                assert n == 0
            except dv.DvError as x:
                assert x.status != dv.DV_ERR_BUFFER_TOO_SMALL, x

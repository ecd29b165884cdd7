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
    assert dv.lib.dv_window_attention(None, 0, n, n, None, 4, 1, None, 0, None) == dv.DV_ERR_INVALID_ARG
    assert dv.lib.dv_window_attention(_cache().ref, 0, n, n, None, 4, 1, None, 0, None) == dv.DV_ERR_INVALID_ARG

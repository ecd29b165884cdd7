"""The operators over the cache without a GPU: what they refuse, before any
pointer is used, and the frequencies of a rotation (CPU)."""
import math

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv

F16 = torch.float16


def _cache(L=2, B=2, H=4, D=64, S=32, P=2):
    return dv.Cache(L, B, H, D, S, P, 0x1000, 0x2000)  # never dereferenced


def _refused(status, fn):
    with pytest.raises(dv.DvError) as ei:
        fn()
    assert ei.value.status == status, ei.value
    return str(ei.value)


S2, E2 = np.array([4, 0], np.int32), np.array([6, 3], np.int32)  # 5 new tokens


def _qo(n=5, heads=8, D=64, dt=F16):
    return torch.zeros(n, heads, D, dtype=dt), torch.zeros(n, heads, D, dtype=dt)


@pytest.mark.parametrize("kind", ["prompt", "tree"])
def test_attention_refusals(kind):
    def call(c=None, layer=0, s=S2, e=E2, q=None, scale=0.125, heads=8, D=64):
        q, o = _qo(int((np.asarray(e) - np.asarray(s)).sum()), heads, D) if q is None else q
        fn = dv.dv_prompt_attention if kind == "prompt" else dv.dv_tree_attention
        fn(c or _cache(), layer, s, e, q, o, scale, None, stream=0)

    _refused(dv.DV_ERR_RANGE, lambda: call(layer=2))
    _refused(dv.DV_ERR_RANGE, lambda: call(layer=-1))
    _refused(dv.DV_ERR_RANGE, lambda: call(layer=2**31 - 1))
    _refused(dv.DV_ERR_RANGE, lambda: call(s=[4, 0], e=[33, 0]))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(heads=6))       # not a multiple of 4 key heads
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(heads=4 * 129))  # a group above 128
    for scale in (0.0, -1.0, math.inf, math.nan):
        _refused(dv.DV_ERR_INVALID_ARG, lambda: call(scale=scale))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(D=136), D=136))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(P=4)))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(P=1)))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(D=60), D=60))
    with pytest.raises(TypeError):
        call(q=_qo(dt=torch.float32))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(q=_qo(n=4)))  # not the ranges' tokens
    with pytest.raises(ValueError):
        call(q=(_qo()[0], _qo(n=4)[1]))
    with pytest.raises(TypeError):  # elements of a head not contiguous
        q = torch.zeros(5, 64, 8, dtype=F16).transpose(1, 2)
        call(q=(q, torch.zeros(5, 8, 64, dtype=F16)))
    call(s=[4, 3], e=[4, 3])  # nothing to do: no pointer is looked at


def test_attention_refuses_more_than_a_tree():
    c = _cache(S=200)
    q, o = _qo(65)
    _refused(dv.DV_ERR_UNSUPPORTED,
             lambda: dv.dv_tree_attention(c, 0, [4, 0], [69, 0], q, o, 0.125, None, stream=0))
    with pytest.raises(ValueError):
        dv.dv_tree_attention(c, 0, S2, E2, *_qo(), 0.125, None, tree=torch.zeros(4, dtype=torch.int64),
                             stream=0)
    with pytest.raises(ValueError):
        dv.dv_tree_attention(c, 0, S2, E2, *_qo(), 0.125, None, tree=torch.zeros(5, dtype=torch.int32),
                             stream=0)


def test_attention_workspace_refusals():
    assert dv.dv_attention_workspace(_cache(), S2, E2, 8) >= 0
    assert dv.dv_attention_workspace(_cache(), [3, 3], [3, 3], 8) == 0
    _refused(dv.DV_ERR_INVALID_ARG, lambda: dv.dv_attention_workspace(_cache(), S2, E2, 6))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: dv.dv_attention_workspace(_cache(), S2, E2, 0))
    _refused(dv.DV_ERR_RANGE, lambda: dv.dv_attention_workspace(_cache(), [0, 0], [33, 0], 8))


def test_append_refusals():
    def call(c=None, layer=0, s=S2, e=E2, q=True, rope=None, positions=None, k=None, q_out=None):
        n = int((np.asarray(e) - np.asarray(s)).sum())
        z = torch.zeros(n, 4, 64, dtype=F16)
        qq = torch.zeros(n, 8, 64, dtype=F16) if q else None
        dv.dv_kv_append(c or _cache(), layer, s, e, z if k is None else k, z, q=qq, q_out=q_out, rope=rope,
                        positions=positions, stream=0)

    _refused(dv.DV_ERR_RANGE, lambda: call(layer=2))
    _refused(dv.DV_ERR_RANGE, lambda: call(s=[31, 0], e=[33, 0]))
    _refused(dv.DV_ERR_UNSUPPORTED, lambda: call(c=_cache(P=4)))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(rope=dv.Rope(128)))  # longer than a head
    bad = dv.Rope(64).c
    bad.rot_dim = 7
    _refused(dv.DV_ERR_INVALID_ARG, lambda: call(rope=bad))
    with pytest.raises(ValueError):
        call(positions=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        call(positions=torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError):
        call(k=torch.zeros(5, 3, 64, dtype=F16))
    with pytest.raises(TypeError):
        call(k=torch.zeros(5, 4, 64))
    call(s=[1, 2], e=[1, 2])


def test_append_refuses_tokens_of_more_than_8m_elements():
    D = (1 << 23) + 8
    k = torch.empty(1, 1, D, dtype=F16)
    _refused(dv.DV_ERR_UNSUPPORTED,
             lambda: dv.dv_kv_append(_cache(L=1, B=1, H=1, D=D, S=4), 0, [0], [1], k, k, stream=0))


def test_compact_refusals():
    keep = torch.zeros(5, dtype=torch.int32)
    _refused(dv.DV_ERR_RANGE, lambda: dv.dv_kv_compact(_cache(), 0, 3, S2, E2, keep, stream=0))
    _refused(dv.DV_ERR_RANGE, lambda: dv.dv_kv_compact(_cache(), 0, 2, [4, 0], [33, 0],
                                                      torch.zeros(29, dtype=torch.int32), stream=0))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: dv.dv_kv_compact(_cache(), 0, 2, S2, E2, keep[:4], stream=0))
    with pytest.raises(ValueError):
        dv.dv_kv_compact(_cache(), 0, 2, S2, E2, keep.long(), stream=0)
    with pytest.raises(TypeError):
        dv.dv_kv_compact(_cache(), 0, 2, S2, E2, torch.zeros(10, dtype=torch.int32)[::2], stream=0)
    dv.dv_kv_compact(_cache(), 0, 2, [1, 2], [1, 2], keep[:0], stream=0)
    dv.dv_kv_compact(_cache(), 1, 1, S2, E2, keep, stream=0)


def test_rope_refusals():
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(rot_dim=64, base=1.0),
               dict(rot_dim=64, base=math.inf), dict(rot_dim=64, scaling="linear", factor=0.5),
               dict(rot_dim=64, scaling="linear", factor=math.nan), dict(rot_dim=2, scaling="ntk", factor=2.0),
               dict(rot_dim=64, scaling="parts", factor=2.0)):
        _refused(dv.DV_ERR_INVALID_ARG, lambda: dv.Rope(**kw))
    _refused(dv.DV_ERR_INVALID_ARG, lambda: dv.dv_rope_init(64, scaling=9))
    with pytest.raises(ValueError):
        dv.Rope(64, scaling="other")


@pytest.mark.parametrize("scaling, factor, original", [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0),
                                                       ("parts", 16.0, 8192)])
@pytest.mark.parametrize("rot, base", [(64, 10000.0), (128, 500000.0), (20, 10000.0), (4, 2.0)])
def test_rope_frequencies(rot, base, scaling, factor, original):
    """turn is f / 2 pi as a 64-bit fraction: both sides are 64-bit floats, each
    a few units of 2^-53 off (pow to one, and a handful of products)."""
    from tests.operator_refs import rope_freqs
    r = dv.Rope(rot, base=base, scaling=scaling, factor=factor, original_max=original).c
    f, m = rope_freqs(rot, base, scaling, factor, original)
    got = np.array([r.turn[i] for i in range(rot // 2)], dtype=np.float64) / 2.0**64
    assert np.all(np.abs(got - f / (2 * math.pi)) <= 2.0**-64 + 16 * 2.0**-53 * f)
    assert abs(r.value_factor - m) <= 2.0**-24 * m
    assert r.rot_dim == rot and all(r.turn[i] == 0 for i in range(rot // 2, dv.DV_MAX_ROT // 2))


def test_null_arguments_from_the_abi():
    c = _cache()
    n = np.zeros(2, np.int32)
    p = n.ctypes.data
    lib = dv.lib
    assert lib.dv_prompt_attention(c.ref, 0, p, p, None, None, 0, None) == dv.DV_ERR_INVALID_ARG
    assert lib.dv_tree_attention(c.ref, 0, p, p, None, None, None, 0, None) == dv.DV_ERR_INVALID_ARG
    assert lib.dv_kv_append(c.ref, 0, p, p, None, None) == dv.DV_ERR_INVALID_ARG
    assert lib.dv_kv_compact(None, 0, 1, p, p, None, 0, None) == dv.DV_ERR_INVALID_ARG
    assert lib.dv_attention_workspace(c.ref, p, p, 4, None) == dv.DV_ERR_INVALID_ARG
    assert lib.dv_rope_init(None, 64, 0, 1e4, 0, 1.0, 0) == dv.DV_ERR_INVALID_ARG

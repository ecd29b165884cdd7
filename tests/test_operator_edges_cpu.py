"""What the operators over the cache refuse by addresses and sizes alone, before any
pointer is looked up (CPU: the tensors here are host memory that no call reaches)."""
import ctypes

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv

F16 = torch.float16


def _refused(status, words, fn):
    with pytest.raises(dv.DvError) as ei:
        fn()
    assert ei.value.status == status and words in str(ei.value), ei.value


class _Case:
    """Two layers of one key head, 8 new tokens of the only sequence, in layer 1."""

    def __init__(self, H=1, D=64, S=64):
        self.K, self.V = (torch.zeros(2, H * D * S, dtype=F16) for _ in range(2))
        self.cache = dv.Cache(2, 1, H, D, S, 2, self.K, self.V)
        self.s, self.e = np.array([8], np.int32), np.array([16], np.int32)
        self.k, self.v, self.q, self.out = (torch.zeros(8, n, D, dtype=F16) for n in (H, H, 2 * H, 2 * H))
        self.positions = torch.zeros(8, dtype=torch.int32)

    def on(self, t, layer, rows=0):
        """[8, 1, D] rows of a layer: with one head, a valid tensor of tokens."""
        return t[layer].view(-1, 1, 64)[rows:rows + 8]

    def append(self, **kw):
        a = dict(k=self.k, v=self.v, q=self.q, q_out=self.out, positions=self.positions) | kw
        dv.dv_kv_append(self.cache, 1, self.s, self.e, a["k"], a["v"], q=a["q"], q_out=a["q_out"],
                        positions=a["positions"], stream=0)


@pytest.mark.parametrize("name", ["k", "v", "q", "q_out", "positions"])
@pytest.mark.parametrize("which", ["K", "V"])
@pytest.mark.parametrize("rows", [0, 8, 40])
def test_append_refuses_to_read_the_layer_it_writes(name, which, rows):
    c = _Case()
    on = c.on(getattr(c, which), 1, rows)
    if name in ("q", "q_out"):
        kw = {"q": torch.zeros(8, 1, 64, dtype=F16), "q_out": torch.zeros(8, 1, 64, dtype=F16)} | {name: on}
    else:
        kw = {name: on.reshape(-1).view(torch.int32)[:8] if name == "positions" else on}
    _refused(dv.DV_ERR_INVALID_ARG, "overlaps the cache's layer", lambda: c.append(**kw))


@pytest.mark.parametrize("name", ["k", "v", "q", "positions"])
def test_append_refuses_to_read_where_it_writes_the_queries(name):
    c = _Case()
    buf = torch.zeros(8 * 2 * 64, dtype=F16)
    kw = {"q_out": buf.view(8, 2, 64)}
    kw |= {"k": dict(k=buf[:8 * 64].view(8, 1, 64)), "v": dict(v=buf[-8 * 64:].view(8, 1, 64)),
           "q": dict(q=buf.view(8, 2, 64)), "positions": dict(positions=buf.view(torch.int32)[100:108])}[name]
    _refused(dv.DV_ERR_INVALID_ARG, "q_out overlaps", lambda: c.append(**kw))


def test_append_takes_another_layers_rows():
    """Past the checks of addresses: what stops it here is that the memory is the host's."""
    c = _Case()
    with pytest.raises(dv.DvError) as ei:
        c.append(k=c.on(c.K, 0), v=c.on(c.V, 0, 40))
    assert "overlaps" not in str(ei.value)


@pytest.mark.parametrize("l0, l1, at, refused", [(0, 2, 0, True), (0, 2, 1, True), (1, 2, 1, True), (1, 2, 0, False)])
@pytest.mark.parametrize("which", ["K", "V"])
def test_compact_refuses_a_list_on_a_layer_it_moves(which, l0, l1, at, refused):
    c = _Case()
    keep = getattr(c, which)[at].view(torch.int32)[200:208]
    with pytest.raises(dv.DvError) as ei:
        dv.dv_kv_compact(c.cache, l0, l1, c.s, c.e, keep, stream=0)
    assert ei.value.status == dv.DV_ERR_INVALID_ARG and ("overlaps" in str(ei.value)) == refused


def test_compact_takes_a_list_between_layers():
    n = 64 * 64
    K, V = (torch.zeros(2, n + 64, dtype=F16) for _ in range(2))
    cache = dv.Cache(2, 1, 1, 64, 64, 2, K, V, layer_stride_elems=n + 64)
    with pytest.raises(dv.DvError) as ei:
        dv.dv_kv_compact(cache, 0, 2, np.array([8]), np.array([16]), K[0, n:n + 16].view(torch.int32), stream=0)
    assert "overlaps" not in str(ei.value)


# ---- sizes that 64 bits do not hold ----------------------------------------------------

FAR = 1 << 40       # elements from one token to the next
MANY = (1 << 23) + 1  # (MANY - 1) * FAR * 2 bytes is 2^64


@pytest.mark.parametrize("name", ["k", "v", "q", "q_out"])
@pytest.mark.parametrize("tokens", [MANY, MANY - 1, 3 * (MANY // 2) + 1])
def test_append_refuses_strides_whose_extent_wraps(name, tokens):
    from kv_cache_streaming_gb300.dv import dv_new_tokens
    c = dv.Cache(1, 1, 1, 8, 1 << 24, 2, 0x1000, 0x2000)
    s, e = np.array([0], np.int32), np.array([tokens], np.int32)
    x = {n: 0x10000000000 * (i + 1) for i, n in enumerate(("k", "v", "q", "q_out"))}
    st = {n: FAR if n == name else 8 for n in x}
    t = dv_new_tokens(dv.DV_DTYPE_FP16, 1, tokens, x["k"], st["k"], x["v"], st["v"], x["q"], st["q"], x["q_out"],
                      st["q_out"], None, None)
    assert dv.lib.dv_kv_append(c.ref, 0, s.ctypes.data, e.ctypes.data, ctypes.byref(t), None) == \
        dv.DV_ERR_BUFFER_TOO_SMALL


@pytest.mark.parametrize("name", ["q", "out"])
def test_attention_refuses_strides_whose_extent_wraps(name):
    from kv_cache_streaming_gb300.dv import dv_queries
    c = dv.Cache(1, 1, 1, 8, 1 << 24, 2, 0x1000, 0x2000)
    s, e = np.array([0], np.int32), np.array([MANY], np.int32)
    a = dv_queries(dv.DV_DTYPE_FP16, 1, MANY, 0x10000000000, FAR if name == "q" else 8, 0x20000000000,
                   FAR if name == "out" else 8, 1.0)
    assert dv.lib.dv_prompt_attention(c.ref, 0, s.ctypes.data, e.ctypes.data, ctypes.byref(a), 0x30000000000,
                                      1 << 40, None) == dv.DV_ERR_BUFFER_TOO_SMALL


@pytest.mark.parametrize("kw", [dict(layer_stride_elems=1 << 60), dict(S=1 << 30, D=1 << 20, B=1 << 10, H=1 << 10)])
def test_caches_whose_bytes_wrap_are_refused(kw):
    g = dict(B=1, H=1, D=64, S=32) | kw
    c = dv.Cache(17, g["B"], g["H"], g["D"], g["S"], 2, 0x1000, 0x2000, layer_stride_elems=g.get("layer_stride_elems", 0))
    s, e = np.zeros(g["B"], np.int32), np.ones(g["B"], np.int32)
    keep = torch.zeros(g["B"], dtype=torch.int32)
    _refused(dv.DV_ERR_UNSUPPORTED, "2^60", lambda: dv.dv_kv_compact(c, 0, 17, s, e, keep, stream=0))


def test_tries_of_a_wait_are_at_most_the_regular_number():
    _refused(dv.DV_ERR_INVALID_ARG, "tries", lambda: dv.dv_debug_attention_tries((1 << 22) + 1))
    dv.dv_debug_attention_tries(1 << 22)
    dv.dv_debug_attention_tries(-5)


# ---- element types -----------------------------------------------------------------------

def _ops(cache, dt):
    s, e = np.array([8], np.int32), np.array([16], np.int32)
    k, q, o = (torch.zeros(8, 1, 64, dtype=dt) for _ in range(3))
    return [lambda: dv.dv_kv_append(cache, 0, s, e, k, k, q=q, q_out=o, stream=0),
            lambda: dv.dv_prompt_attention(cache, 0, s, e, q, o, 0.125, None, stream=0),
            lambda: dv.dv_tree_attention(cache, 0, s, e, q, o, 0.125, None, stream=0)]


@pytest.mark.parametrize("op", range(3))
@pytest.mark.parametrize("held, given", [(torch.float16, torch.bfloat16), (torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("which", ["K", "V", "both"])
def test_tokens_of_another_float_type_than_the_caches_are_refused(op, held, given, which):
    K, V = (torch.zeros(64 * 64, dtype=held if which in (n, "both") else given) for n in "KV")
    with pytest.raises(TypeError, match="the cache's tensors are"):
        _ops(dv.Cache(1, 1, 1, 64, 64, 2, K, V), given)[op]()


@pytest.mark.parametrize("op", range(3))
@pytest.mark.parametrize("kind", ["same", "bytes", "int16", "float32", "addresses"])
def test_caches_of_other_words_take_either_type(op, kind):
    """Memory whose dtype says nothing of its elements (the call goes on to the pointers)."""
    for dt in (torch.float16, torch.bfloat16):
        n = {"bytes": (torch.uint8, 2), "int16": (torch.int16, 1), "float32": (torch.float32, 1)}.get(kind, (dt, 1))
        K, V = (torch.zeros(64 * 64 * n[1], dtype=n[0]) for _ in "KV")
        if kind == "addresses":
            K, V = 0x10000000, 0x20000000
        with pytest.raises(dv.DvError):
            _ops(dv.Cache(1, 1, 1, 64, 64, 2, K, V), dt)[op]()

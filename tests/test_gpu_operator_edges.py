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

"""Attention beside rows whose look takes long: non-finite values in rows that a mask hides are taken out
of each tile in shared memory before its product, value by value, while the chains of products
go on to other tiles and units.  No tile may be multiplied before it has come and been
looked at, however late the look is: many short units in a row, of which the last (or first) tiles
hold such rows and the ones between do not."""
import math

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv
from tests import bounded_refs as W
from tests import operator_refs as R
from tests import test_gpu_window as window

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    dv.dv_attention_check()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ws(cache, s, e, heads, size=dv.dv_attention_workspace):
    return torch.full((size(cache, s, e, heads),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("B, H, D, ctx, new, rows, sinks", [
    (34, 27, 64, 408, 41, 333, 1),   # the first half of a unit's first tile hidden but for one row
    (34, 40, 64, 430, 8, 300, 4),
    (20, 64, 128, 900, 20, 400, 1),
    (40, 31, 128, 700, 3, 260, 33),
])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_windows_of_many_units(dtype, B, H, D, ctx, new, rows, sinks):
    window.test_window_attention(dtype, B, H, 1, D, ctx + new + 8, (0, ctx), (1, new), rows, sinks)
    window.test_window_attention(dtype, B, H, 1, D, ctx + new + 9, (ctx - 60, ctx), (1, new), rows, sinks)


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_units_of_two_and_three_tiles_in_turn(dtype, D, scored):
    """Trees whose nodes attend the context and the first node alone; the other nodes' rows, in each
    unit's last tile, hold NaN.  Scored: one token, the rows past it."""
    B, n, S = 608, 64, 400
    gen = _gen(D)
    s = np.where(np.arange(B) % 2 == 0, 188, 316).astype(np.int32)
    e = (s + (1 if scored else n)).astype(np.int32)
    cache, K, V = R.make_cache(dtype, 1, B, 1, D, S, gen)
    q = torch.empty(int((e - s).sum()), 1, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) * 2
    for b in range(B):
        V[0, b, 0, s[b] + 1:] = (math.nan, math.inf, -math.inf)[b % 3]
        K[0, b, 0, :, s[b] + 1:] = math.nan
    out = torch.full_like(q, math.nan)
    if scored:
        mass = torch.zeros(B, 1, S, device="cuda")
        want, tol, m, mtol = W.attend_ref(K[0], V[0], s, e, q, 0.1, mass=mass)
        dv.dv_scored_attention(cache, 0, s, e, q, out, 0.1, mass, _ws(cache, s, e, 1, dv.dv_scored_attention_workspace))
        R.assert_within(mass, m, mtol, "weights")
    else:
        masks = [(torch.arange(z, device="cuda") <= a).expand(n, z) for a, z in zip(s.tolist(), e.tolist())]
        want, tol, _, _ = W.attend_ref(K[0], V[0], s, e, q, 0.1, masks=masks)
        tree = R.bits_tensor([1] * int(q.shape[0]))
        dv.dv_tree_attention(cache, 0, s, e, q, out, 0.1, _ws(cache, s, e, 1), tree=tree)
    assert bool(want.isfinite().all())
    R.assert_within(out, want, tol)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prompts_whose_last_rows_are_not_numbers(dtype, D):
    """Two row tiles a unit: the second's last tile, which the first does not attend, holds NaN for the
    last tokens; the units that follow begin with tiles of the context."""
    B, H, S = 6, 100, 470
    gen = _gen(D + 1)
    s = np.full(B, 256, np.int32)
    e = (s + np.array([200, 190, 200, 180, 200, 150])).astype(np.int32)
    cache, K, V = R.make_cache(dtype, 1, B, H, D, S, gen)
    q = torch.empty(int((e - s).sum()), H, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) * 2
    for b in range(B):
        V[0, b, :, 392:] = math.nan
        V[0, b, ::2, 385:392] = math.inf
    out = torch.full_like(q, math.nan)
    want, tol = R.attention_ref(K[0], V[0], s, e, q, 0.1)
    dv.dv_prompt_attention(cache, 0, s, e, q, out, 0.1, _ws(cache, s, e, H))
    assert bool(want.isnan().any()) and int(want.isfinite().sum()) > want.numel() // 2
    R.assert_within(out, want, tol)

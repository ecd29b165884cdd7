"""The speculative decoding example: its tokens are plain greedy decoding's, its rows
of the cache are what decoding token by token writes (to rounding), and the host
replica restores them."""
import importlib.util
from pathlib import Path

import pytest
import torch

import kv_cache_streaming_gb300 as dv

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parent.parent


def test_speculative_example_decodes_as_plain_decoding_does():
    spec = importlib.util.spec_from_file_location("speculative", ROOT / "examples" / "speculative.py")
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    prompts, tree, plain = ex.main(steps=40)
    assert tree["tokens"] == plain["tokens"]
    assert tree["steps"] < plain["steps"]  # some drafts were taken
    shape_k, shape_v = (ex.L, ex.B, ex.H, ex.D // 8, ex.S, 8), (ex.L, ex.B, ex.H, ex.S, ex.D)
    for b, p in enumerate(prompts):
        n = len(p) + 39  # rows of the prompt and of all generated tokens but the last
        for name, shape, dim in (("k", shape_k, 3), ("v", shape_v, 2)):
            a, z = (getattr(r["model"], name).view(shape)[:, b].narrow(dim, 0, n).double() for r in (tree, plain))
            # fp16 activations of a few layers: a few half steps of 2^-11 on values of order one
            assert float((a - z).abs().max()) < 2.0 ** -5
    # the replica holds every kept row
    m = tree["model"]
    back = dv.Cache(ex.L, ex.B, ex.H, ex.D, ex.S, 2, torch.zeros_like(m.k), torch.zeros_like(m.v))
    tree["replica"].restore_batched(back)
    torch.cuda.synchronize()
    for b, n in enumerate(tree["lens"].tolist()):
        for t, u, shape, dim in ((m.k, back.k, shape_k, 3), (m.v, back.v, shape_v, 2)):
            assert torch.equal(t.view(shape)[:, b].narrow(dim, 0, n), u.view(shape)[:, b].narrow(dim, 0, n))
    dv.dv_attention_check()

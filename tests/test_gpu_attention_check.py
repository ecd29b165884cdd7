"""What dv_attention_check costs: it fetches the counts of the attention forms that the process
has launched, and of no others (whose kernels a fetch would load).  In a process of its own."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = """
import numpy as np, torch
from torch.profiler import ProfilerActivity, profile
import kv_cache_streaming_gb300 as dv

B, H, D, S = 2, 2, 64, 130
k, v = (torch.ones(B * H * D * S, dtype=torch.bfloat16, device="cuda") for _ in range(2))
cache = dv.Cache(1, B, H, D, S, 2, k, v)
e = np.full(B, S, np.int32)
s = e - 1
q = torch.ones(B, H, D, dtype=torch.bfloat16, device="cuda")
out = torch.empty_like(q)
mass = torch.zeros(B, H, S, device="cuda")
ws = torch.empty(dv.dv_scored_attention_workspace(cache, s, e, H), dtype=torch.uint8, device="cuda")
forms = [lambda: None, lambda: dv.dv_tree_attention(cache, 0, s, e, q, out, 0.125, ws),
         lambda: dv.dv_window_attention(cache, 0, s, e, q, out, 0.125, 100, 4, ws),
         lambda: dv.dv_scored_attention(cache, 0, s, e, q, out, 0.125, mass, ws)]

def fetches(call):
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    return sum("DtoH" in x.name for x in prof.events())

fetches(lambda: out.cpu())  # (a process's first recording may miss some)
seen = [fetches(lambda: out.cpu())]
for form in forms:
    form()
    torch.cuda.synchronize()
    seen.append(fetches(dv.dv_attention_check))
assert float(out.float().mean()) == 1.0
print("fetches", *seen)
"""


def test_only_forms_that_were_launched_are_asked():
    root = Path(__file__).resolve().parent.parent
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    line = next(x for x in r.stdout.splitlines() if x.startswith("fetches"))
    control, *seen = map(int, line.split()[1:])
    if control != 1:
        pytest.skip("the profiler records no copies here")
    assert seen == [0, 1, 2, 3]

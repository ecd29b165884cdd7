"""Rotary frequencies against values worked out apart from the library: in 50 decimal
digits and from wavelengths, and for given frequencies as models are run with them."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import kv_cache_streaming_gb300 as dv
from tests import operator_refs as R

getcontext().prec = 50
PI = Decimal("3.14159265358979323846264338327950288419716939937511")


def wavelengths(rot, base, scaling, factor, original):
    """Positions that each pair takes for a turn, by the cases of the paper: a wavelength of
    which 32 or more fit the trained context stays, one of which at most one fits is stretched by
    the factor, those between are mixed as frequencies."""
    base, factor, out = Decimal(base), Decimal(factor), []
    if scaling == "ntk":
        # the slowest pair is stretched by the factor, the fastest not at all
        base *= (factor.ln() * Decimal(rot) / Decimal(rot - 2)).exp()
    for i in range(rot // 2):
        w = 2 * PI * (base.ln() * Decimal(2 * i) / Decimal(rot)).exp()
        if scaling == "linear":
            w *= factor
        if scaling == "parts":
            fit = Decimal(original) / w
            if fit <= 1:
                w *= factor
            elif fit < 32:
                keep = (fit - 1) / 31
                w = 1 / (keep / w + (1 - keep) / (w * factor))
        out.append(w)
    return out


@pytest.mark.parametrize("scaling, factor, original", [("none", 1, 0), ("linear", 4, 0), ("ntk", 8, 0),
                                                       ("parts", 16, 4096), ("parts", 4, 32768)])
@pytest.mark.parametrize("rot, base", [(64, 10000), (128, 500000), (20, 10000), (256, 1000000)])
def test_frequencies_from_wavelengths(rot, base, scaling, factor, original):
    r = dv.Rope(rot, base=float(base), scaling=scaling, factor=float(factor), original_max=original).c
    for i, w in enumerate(wavelengths(rot, base, scaling, factor, original)):
        # a few roundings of 64-bit floats, and the fraction's last place
        assert abs(Decimal(r.turn[i]) / 2 ** 64 - 1 / w) <= Decimal(2) ** -64 + Decimal(2) ** -48 / w
    m = float(Decimal(factor).ln() / 10 + 1) if scaling == "parts" else 1.0
    assert abs(r.value_factor - m) <= 2.0 ** -24 * m


def test_known_frequencies():
    """By hand: base 10000 and 4 rotated elements are 1 and 1/100 radians a position; a context of
    100 turns of the first pair and one of the second leaves the one and stretches the other."""
    r = dv.Rope(4, base=10000.0).c
    assert [r.turn[i] / 2.0 ** 64 for i in range(2)] == pytest.approx([0.15915494309189535, 0.0015915494309189535], rel=1e-15)
    r = dv.Rope(4, base=10000.0, scaling="parts", factor=8.0, original_max=628).c
    assert [r.turn[i] / 2.0 ** 64 for i in range(2)] == pytest.approx([0.15915494309189535, 0.0001989436788648692], rel=1e-15)


def by_index(rot, base, factor, original, fast=32.0, slow=1.0):
    """Frequencies as models scaled by parts are commonly run: a ramp over the pairs' indices between
    the rounded ones at which `fast` and `slow` turns fit the trained context."""
    def index(turns):
        return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(index(fast))), min(rot - 1, math.ceil(index(slow)))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot // 2)]
    return [x * (1 - g) + x / factor * g for x, g in zip(f, ramp)]


def test_given_frequencies_become_turns():
    f = by_index(128, 10000.0, 16.0, 4096)
    r = dv.Rope.from_frequencies(f, interleaved=True, value_factor=0.5).c
    assert (r.rot_dim, r.interleaved, r.value_factor) == (128, 1, 0.5)
    for i, x in enumerate(f):
        assert abs(Decimal(r.turn[i]) / 2 ** 64 - Decimal(x) / (2 * PI)) <= Decimal(2) ** -64 + Decimal(2) ** -50 * Decimal(x)
    assert all(r.turn[i] == 0 for i in range(64, dv.DV_MAX_ROT // 2))
    # the two ramps do differ, as documented
    theirs = dv.Rope(128, scaling="parts", factor=16.0, original_max=4096).c
    assert max(abs(r.turn[i] / theirs.turn[i] - 1) for i in range(64)) > 0.5


def test_given_frequencies_that_are_refused():
    for f in ([], [1.0] * 129, [1.0, math.nan], [math.inf]):
        with pytest.raises(ValueError):
            dv.Rope.from_frequencies(f)
    c = dv.Cache(1, 1, 1, 64, 64, 2, 0x10000000, 0x20000000)
    k = torch.zeros(8, 1, 64, dtype=torch.float16)
    for factor in (math.nan, math.inf):
        with pytest.raises(dv.DvError) as ei:
            dv.dv_kv_append(c, 0, [0], [8], k, k, rope=dv.Rope.from_frequencies([1.0], value_factor=factor), stream=0)
        assert ei.value.status == dv.DV_ERR_INVALID_ARG and "value_factor" in str(ei.value)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("new", [1, 40])
def test_append_with_given_frequencies(dtype, inter, new):
    B, H, D, rot = 2, 3, 128, 96
    gen = torch.Generator(device="cuda").manual_seed(new)
    f = np.array(by_index(rot, 10000.0, 16.0, 4096))
    f[-1] = -f[-1]  # turning the other way is a frequency too
    s = np.array([3, 0], np.int32)
    e = s + new
    cache, K, V = R.make_cache(dtype, 1, B, H, D, 64, gen)
    q, k, v = (torch.empty(B * new, H, D, dtype=R.DT[dtype], device="cuda").normal_(generator=gen) for _ in range(3))
    pos = torch.randint(0, 1 << 18, (B * new,), generator=gen, device="cuda", dtype=torch.int32)
    rope = dv.Rope.from_frequencies(f, interleaved=inter, value_factor=1.25)
    got = dv.dv_kv_append(cache, 0, s, e, k, v, q=q, rope=rope, positions=pos)
    want, tol = R.rotate_ref(q, pos, rot, inter, f, 1.25)
    R.assert_within(got[..., :rot], want[..., :rot], tol[..., :rot])
    assert torch.equal(got[..., rot:], q[..., rot:])
    want, tol = R.rotate_ref(k, pos, rot, inter, f, 1.25)
    rows = torch.cat([K[0, b, :, :, a:z].permute(2, 0, 1, 3).reshape(z - a, H, D) for b, _, a, z in R.spans(s, e)])
    R.assert_within(rows[..., :rot], want[..., :rot], tol[..., :rot])

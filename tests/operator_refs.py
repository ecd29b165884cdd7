"""Plain 64-bit forms of the operators over the cache, for their tests, with the
error bounds that the kernels' roundings allow (derived beside each)."""
from __future__ import annotations

import math

import numpy as np
import torch

import kv_cache_streaming_gb300 as dv

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    """The most a rounding to `dtype` is off, relative to the value."""
    return torch.finfo(dtype).eps / 2


def make_cache(dtype, L, B, H, D, S, gen, fill=None, stride=0):
    """(dv.Cache, K [L, B, H, D/8, S, 8], V [L, B, H, S, D]); layers `stride`
    elements apart (0: densely)."""
    stride = stride or B * H * D * S
    k = torch.empty(L, stride, dtype=DT[dtype], device="cuda")
    v = torch.empty(L, stride, dtype=DT[dtype], device="cuda")
    for t in (k, v):
        if fill is None:
            t.normal_(generator=gen)
        else:
            t.fill_(fill)
    cache = dv.Cache(L, B, H, D, S, 2, k, v, layer_stride_elems=stride)
    n = B * H * D * S
    return cache, k[:, :n].view(L, B, H, D // 8, S, 8), v[:, :n].view(L, B, H, S, D)


def spans(s, e):
    t = 0
    for b, (a, z) in enumerate(zip(np.asarray(s).tolist(), np.asarray(e).tolist())):
        yield b, t, a, z
        t += z - a


def attended(a, z, bits, device="cuda"):
    """[n, z] truth values of one sequence: causal, or the context and the
    tree's bits (a list of Python integers)."""
    n = z - a
    ok = torch.zeros(n, z, dtype=torch.bool)
    ok[:, :a] = True
    for i in range(n):
        if bits is None:
            ok[i, a:a + i + 1] = True
        else:
            for j in range(n):
                ok[i, a + j] = bool(bits[i] >> j & 1)
    return ok.to(device)


def attention_ref(K, V, s, e, q, scale, bits=None):
    """(outputs, error bounds) in 64 bits, [T, Hq, D].  K, V: one layer.

    The bound, with u = half a step of the type, w the exact weights and
    A = sum_j w_j |v_j|:
      u A             weights rounded to the type before the product with V
      2 ds A          each score is off by at most ds = D 2^-24 max_j sum_d |q_d k_jd| scale
                      (products of 16-bit values are exact in 32 bits, their sum is not), the
                      weight by twice that (itself and the normalisation)
      (2^-21 + (n+8) 2^-24) A   exp2 and its argument's rounding; 32-bit sums over n rows
      u |o|           the output's own rounding (and 2^-25 below fp16's smallest normal)
      2^-25 sum|v|    fp16: weights below 2^-14 of the largest lose relative precision."""
    dt = q.dtype
    u = half_step(dt)
    H = K.shape[1]
    G, D = q.shape[1] // H, q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for b, t, a, z in spans(s, e):
        n = z - a
        if n == 0:
            continue
        ok = attended(a, z, None if bits is None else bits[t:t + n])
        for h in range(H):
            k = K[b, h, :, :z].double().transpose(0, 1).reshape(z, D)
            v = V[b, h, :z].double()
            qq = q[t:t + n, h * G:(h + 1) * G].double()
            x = torch.einsum("ngd,kd->ngk", qq, k) * scale
            seen = ok[:, None, :]
            x = torch.where(seen, x, -math.inf)
            m = x.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            w = torch.exp(x - m)
            tot = w.sum(-1, keepdim=True)
            w = torch.where(tot == 0, 0.0, w / tot)
            if torch.isfinite(v).all():
                o = torch.einsum("ngk,kd->ngd", w, v)
            else:  # rows that are not attended have no part in the sum, whatever they hold
                vv = torch.where(ok[..., None], v[None], 0.0)
                o = torch.einsum("ngk,nkd->ngd", w, vv)
            va = torch.nan_to_num(v.abs(), nan=0.0, posinf=0.0)
            A = torch.einsum("ngk,kd->ngd", w, va)
            ka = torch.nan_to_num(k.abs(), nan=0.0, posinf=0.0)
            qk = torch.where(seen, torch.einsum("ngd,kd->ngk", qq.abs(), ka), 0.0).amax(-1, keepdim=True)
            ds = D * 2.0 ** -24 * qk * scale
            bound = A * (u + 2 * ds + 2.0 ** -21 + (z + 8) * 2.0 ** -24) + u * o.abs() + 2.0 ** -25
            if dt == torch.float16:
                bound = bound + 2.0 ** -25 * va.sum(0)
            out[t:t + n, h * G:(h + 1) * G] = o
            tol[t:t + n, h * G:(h + 1) * G] = bound
    return out, tol


def assert_within(got, want, tol, what=""):
    got = got.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~nan & ~inf
    err = (got[ok] - want[ok]).abs() - tol[ok]
    bad = err > 0
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {err.numel()} outside the bound, by up to " \
                                f"{float(err.max()):.3g}"


def random_tree(n, rng):
    """(bits, depth) of a random tree of n nodes, parents first."""
    bits, depth = [], []
    for i in range(n):
        p = int(rng.integers(max(0, (i - 1) // 3), i)) if i else -1
        bits.append((bits[p] if i else 0) | 1 << i)
        depth.append(depth[p] + 1 if i else 0)
    return bits, depth


def bits_tensor(bits):
    return torch.from_numpy(np.array(bits, np.uint64).view(np.int64)).cuda()


def rope_freqs(rot, base, scaling, factor, original):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        g = np.clip((original * f / (2 * math.pi) - 1) / 31, 0, 1)
        return g * f + (1 - g) * f / factor, 0.1 * math.log(factor) + 1
    return f, 1.0


def rotate_ref(x, pos, rot, interleaved, freqs, factor):
    """(values, bounds) in 64 bits of x [T, heads, D] rotated at pos [T].

    The bound: half a step of the type on the result (2^-25 below fp16's
    normals), and (|x| + |y|) m times 2^-20 for what is done in 32 bits: the
    angle's rounding (pi 2^-25), sine and cosine to 2 units of 2^-24 each, two
    products and a sum."""
    u = half_step(x.dtype)
    w, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None] * torch.from_numpy(freqs).to(x.device)
    c, s = (torch.cos(ang) * factor)[:, None], (torch.sin(ang) * factor)[:, None]
    i = torch.arange(rot // 2, device=x.device)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., one].double(), x[..., two].double()
    w[..., one], w[..., two] = a * c - b * s, a * s + b * c
    both = (a.abs() + b.abs()) * factor * 2.0 ** -20
    for at in (one, two):
        tol[..., at] = u * w[..., at].abs() + both + 2.0 ** -25
    return w, tol

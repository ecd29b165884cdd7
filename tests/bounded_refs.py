"""Plain 64-bit forms of the operators that keep a cache within a bound, for their
tests, with the error bounds that the kernels' roundings allow."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.operator_refs import half_step, spans


def window_mask(a, z, window=1 << 40, sinks=0, device="cuda"):
    """[z - a, z] truth values: which rows the tokens at rows [a, z) attend."""
    r, j = torch.arange(a, z, device=device)[:, None], torch.arange(z, device=device)
    return (j <= r) & ((j > r - window) | (j < sinks))


def weights_ref(k, q, ok, scale):
    """(weights, bounds on their relative error) in 64 bits of one key head: k [z, D],
    q [n, G, D], ok [n, z]; weights [n, G, z], bounds [n, G, 1].

    The bound: 2 ds, with ds = D 2^-24 max_j sum_d |q_d k_jd| scale the most a score is off
    (products of 16-bit values are exact in 32 bits, their sum is not), for the weight itself
    and the normalisation; 2^-21 for exp2 and log2; z + 8 roundings of the 32-bit sum of
    weights; and the rounding, to 32 bits, of the statistic max + log2(sum) and of what the
    exponent is taken of: 2^-23 of the largest score in log2 units, twice."""
    x = torch.einsum("ngd,kd->ngk", q.double(), k.double()) * scale
    seen = ok[:, None, :]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    w = w / w.sum(-1, keepdim=True)
    w = torch.where(seen.any(-1, keepdim=True), w, 0.0)
    qk = torch.einsum("ngd,kd->ngk", q.double().abs(), torch.nan_to_num(k.double().abs(), nan=0.0, posinf=0.0))
    qk = torch.where(seen, qk, 0.0).amax(-1, keepdim=True) * scale
    z, D = k.shape
    return w, 2 * D * 2.0 ** -24 * qk + 2.0 ** -21 + (z + 8) * 2.0 ** -24 + 2 * 2.0 ** -23 * (qk * 1.45 + 2 * math.log2(z + 1))


def attend_ref(K, V, s, e, q, scale, window=1 << 40, sinks=0, last=0, mass=None, masks=None):
    """(outputs, bounds, mass, bounds) in 64 bits; K, V: one layer; q [T, Hq, D]; mass
    [B, H, S] (or None), to which the weights of the last `last` tokens (0: all) are added; masks:
    what the tokens of each sequence attend, [z - a, z] (None: by the window).

    Outputs, with u half a step of the type and A = sum_j w_j |v_j|: u A for the weights'
    rounding to the type before the product with V, weights_ref's bound times A (its sum
    of weights and the product's over z rows), u |o| for the output's own rounding, 2^-25 below
    fp16's smallest normal; fp16 holds weights below 2^-21 of the largest with fewer bits:
    2^-25 sum |v|.  Mass: weights_ref's bound times what is added, and a 32-bit rounding of
    the total for each of the added weights' partial sums (at most one a weight, of at most
    the final sum) and for the last addition."""
    dt, u = q.dtype, half_step(q.dtype)
    H = K.shape[1]
    G, D = q.shape[1] // H, q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    m64 = None if mass is None else mass.double().clone()
    mtol = None if mass is None else torch.zeros_like(m64)
    for b, t, a, z in spans(s, e):
        n = z - a
        if n == 0:
            continue
        ok = window_mask(a, z, window, sinks, q.device) if masks is None else masks[b]
        counted = n if last == 0 else min(n, last)
        for h in range(H):
            k = K[b, h, :, :z].transpose(0, 1).reshape(z, D)
            v = V[b, h, :z].double()
            w, rel = weights_ref(k, q[t:t + n, h * G:(h + 1) * G], ok, scale)
            if torch.isfinite(v).all():
                o = torch.einsum("ngk,kd->ngd", w, v)
            else:  # rows that are not attended have no part in the sum, whatever they hold
                o = torch.einsum("ngk,nkd->ngd", w, torch.where(ok[..., None], v[None], 0.0))
            va = torch.nan_to_num(v.abs(), nan=0.0, posinf=0.0)
            A = torch.einsum("ngk,kd->ngd", w, va)
            bound = A * (u + rel) + u * o.abs() + 2.0 ** -25
            if dt == torch.float16:
                bound = bound + 2.0 ** -25 * torch.einsum("nk,kd->nd", ok.double(), va)[:, None]
            out[t:t + n, h * G:(h + 1) * G], tol[t:t + n, h * G:(h + 1) * G] = o, bound
            if mass is not None:
                wc, rc = w[n - counted:], rel[n - counted:]
                add = wc.sum((0, 1))
                err = (wc * rc).sum((0, 1)) + add * (counted * G * 2.0 ** -24)
                seen = ok[n - counted:].any(0)
                m64[b, h, :z] += torch.where(seen, add, 0.0)
                mtol[b, h, :z] = torch.where(seen, err + 2.0 ** -23 * m64[b, h, :z].abs(), 0.0)
    return out, tol, m64, mtol


def evict_rows(mass, rows, kept, sinks, recent):
    """The rows that stay of each (layer, head, sequence), [L][H][B] lists: a sort by (weight
    from above, row), NaN above all numbers.  mass: [L, B, H, S], any device."""
    m = mass.detach().cpu().double().numpy()
    out = []
    for l in range(m.shape[0]):
        out.append([])
        for h in range(m.shape[2]):
            lists = []
            for b, (n, k) in enumerate(zip(rows.tolist(), kept.tolist())):
                if n == k:
                    lists.append(list(range(n)))
                    continue
                x = m[l, b, h]
                mid = sorted(range(sinks, n - recent), key=lambda i: (-math.inf if math.isnan(x[i]) else -x[i],
                                                                      not math.isnan(x[i]), i))
                top = sorted(mid[:k - sinks - recent])
                lists.append(list(range(sinks)) + top + list(range(n - recent, n)))
            out[-1].append(lists)
    return out

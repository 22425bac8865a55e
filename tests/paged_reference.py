"""The paged-cache operators' definitions in 64 bits (numpy), one loop per
definition, and the error bounds that the GPU results are held to.

Half a step of a type is eps / 2 relative to the value: 2^-8 for bf16, 2^-24 for
fp32.  F is that of fp32, in which everything is computed."""
from __future__ import annotations

import math

import numpy as np

F = 2.0 ** -24
STEP = {"bf16": 2.0 ** -8, "f32": F}


# ------------------------------------------------------------------ plan --

def plan(lens, new, free, count, table, page, n_slots, release=None):
    """Sequence by sequence.  free: the stack's array, count its entries.
    Returns a dict of lists; table and free come back changed."""
    B, M = len(lens), len(table[0])
    table, free, lens = [list(r) for r in table], list(free), list(lens)
    if release is not None:
        for b in range(B):
            if release[b]:
                for j in range(-(-lens[b] // page)):
                    free[count] = table[b][j]
                    count += 1
                lens[b] = 0
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    slot, pos = [-1] * n_slots, [0] * n_slots
    granted, out, demand, taken = [0] * B, list(lens), 0, 0
    for b in range(B):
        held, want = -(-lens[b] // page), -(-(lens[b] + new[b]) // page)
        fits = lens[b] + new[b] <= M * page and cu[b + 1] <= n_slots
        need = want - held if fits else 0
        at = demand
        demand += need
        if fits and (need == 0 or demand <= count):
            granted[b] = new[b]
            for i in range(need):
                table[b][held + i] = free[count - 1 - at - i]
            taken += need
        out[b] = lens[b] + granted[b]
        for t in range(cu[b], min(cu[b + 1], n_slots)):
            p = lens[b] + t - cu[b]
            pos[t] = p
            if granted[b]:
                slot[t] = table[b][p // page] * page + p % page
    return dict(lens=out, free_count=[count - taken], cu_tokens=cu, granted=granted, slot=slot,
                pos=pos, table=table, free=free)


# ------------------------------------------------------------- rotation --

def rates(R, theta, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    w = theta ** (-2.0 * np.arange(R // 2) / max(R, 1))
    if scaling == "linear":
        return w / factor
    if scaling == "yarn":
        def at(turns):
            return R * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(theta))
        lo, hi = max(0, math.floor(at(beta_fast))), min(R - 1, math.ceil(at(beta_slow)))
        g = np.clip((np.arange(R // 2) - lo) / (hi - lo if hi != lo else 0.001), 0, 1)
        return w * (1 - g) + w / factor * g
    return w


def magnitude(scaling="none", factor=1.0, magnitude=0.0, **_):
    return magnitude or (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)


def members(R, layout):
    """(first, second) dimension of every pair."""
    i = np.arange(R // 2)
    return (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rotate(x, pos, R, layout, w, m, back=False):
    """x [tokens, H, D] rotated by pos (back: by the transpose)."""
    y = x.copy()
    if R == 0:
        return y
    a, b = members(R, layout)
    ang = pos[:, None, None] * w
    c, s = np.cos(ang) * m, np.sin(ang) * m * (-1 if back else 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, weight, pos, R, layout, w, m, eps, dtype):
    """(y, bound): the result and the error an fp32 evaluation rounded once to
    dtype may have.

    r: a sum of D <= 128 squares in chains of at most 8 and 5 tree levels, so at
    most 13 roundings of sums and 1 of each square, halved by the root, and the
    root's own 2 steps: 9 F.  cos, sin: the angle to pi F, the function to 2 F.
    The constants w cos and w sin, three products and a sum, two roundings of
    weight and mean: 7 more.  24 F of the sum of the magnitudes covers them."""
    n = x.copy()
    if weight is not None:
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    y = rotate(n, pos, R, layout, w, m)
    mag = np.abs(n)
    if R:
        a, b = members(R, layout)
        both = (mag[..., a] + mag[..., b]) * m
        mag[..., a], mag[..., b] = both, both
    return y, 24 * F * mag + STEP[dtype] * np.abs(y)


def norm_rope_grad(x, dy, weight, pos, R, layout, w, m, eps, dtype):
    """((dx, bound), (dw, bound)); the second None without a weight.

    g carries the 24 F of the rotation; u = g w, the mean of u x (13 roundings of
    sums, 3 of products) and r^3 (3 times 9 F, 4 products) add at most 64 F of the
    magnitudes of the two terms.  dw is a sum of one term per token and head, each
    good to 64 F, in chains of at most `chain` additions: a warp's lane adds its
    rows one after the other, then 2 to 4 tree levels, 8 warps, ceil(CTAs / 32) <= 10
    and 5 levels."""
    g = rotate(dy, pos, R, layout, w, m, back=True)
    gm = np.abs(dy).copy()
    if R:
        a, b = members(R, layout)
        both = (gm[..., a] + gm[..., b]) * m
        gm[..., a], gm[..., b] = both, both
    if weight is None:
        return (g, 24 * F * gm + STEP[dtype] * np.abs(g)), None
    D = x.shape[-1]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = g * weight
    dx = r * u - x * r ** 3 * (u * x).mean(-1, keepdims=True)
    um = gm * np.abs(weight)
    bound = 64 * F * (r * um + np.abs(x) * r ** 3 * (um * np.abs(x)).sum(-1, keepdims=True) / D)
    dw = (g * x * r).sum((0, 1))
    terms = (gm * np.abs(x) * r).sum((0, 1))
    chain = x.shape[0] * x.shape[1] / 32 + 64
    return (dx, bound + STEP[dtype] * np.abs(dx)), (dw, (64 + chain) * F * terms)


# --------------------------------------------------------------- decode --

def visible(n, window, sinks):
    return [j for j in range(n) if window == 0 or j >= n - window or j < sinks]


def decode(q, k_pages, v_pages, table, lens, window, sinks, dtype, scale=None, skip=()):
    """(out, lse, bound of out, bound of lse).  skip: page ids left out.

    delta: what D products and sums in fp32 (any order) may change a score by, plus
    the rounding of scale and score (8 F of it).  A weight is off by 2 delta (its own
    score and the reference), ex2 2^-22, for bf16 its rounding; sums over n keys by
    n + 64 roundings at most; the output is rounded once."""
    B, Hq, D = q.shape
    page, Hkv = k_pages.shape[1:3]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    bo, bl = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        toks = [j for j in visible(int(lens[b]), window, sinks) if int(table[b][j // page]) not in skip]
        if not toks:
            continue
        rows = [(int(table[b][j // page]), j % page) for j in toks]
        k = np.stack([k_pages[p, o] for p, o in rows])
        v = np.stack([v_pages[p, o] for p, o in rows])
        n = len(toks)
        for h in range(Hq):
            kk, vv = k[:, h // G], v[:, h // G]
            s = kk @ q[b, h] * scale
            delta = ((D + 8) * F * (np.abs(kk) @ np.abs(q[b, h])) * scale + 8 * F * np.abs(s)).max()
            top = s.max()
            p = np.exp(s - top)
            z = p.sum()
            out[b, h] = p @ vv / z
            lse[b, h] = top + np.log(z)
            mag = p @ np.abs(vv) / z
            rel = 2 * delta + 2 ** -22 + (n + 64) * F
            bo[b, h] = (2 * rel + (STEP["bf16"] if dtype == "bf16" else 0)) * mag \
                + STEP[dtype] * np.abs(out[b, h])
            bl[b, h] = rel + 4 * F * abs(lse[b, h])
    return out, lse, bo, bl


def worst(got, want, bound):
    """The largest error in units of its bound; infinite where only one is finite."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.where(same, 0.0, np.abs(got - want) / np.maximum(bound, 1e-300))
    return float(np.nan_to_num(e, nan=np.inf).max()) if e.size else 0.0

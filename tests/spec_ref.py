"""Plain 64-bit (and exact rational) implementations of the rotary, verification and commit calls,
straight from their definitions in include/infllmv2.h."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


def turn_fraction(freqs: np.ndarray, pos: np.ndarray) -> np.ndarray:
    """Angle in radians of each (position, pair) from the table of uint64 turns, by exact integers."""
    out = np.empty((len(pos), len(freqs)))
    for r, x in enumerate(pos):
        for i, f in enumerate(freqs):
            out[r, i] = 2.0 * math.pi * (((int(x) * int(f)) % (1 << 64)) / 2.0 ** 64)
    return out


def rotate(x: np.ndarray, angle: np.ndarray, rot: int, interleaved: bool, scale: float = 1.0, transposed: bool = False):
    """x [rows, heads, d] in fp64 turned by angle [rows, rot/2]; also returns |a| + |b| per element
    (what an error of the factors is multiplied by; 0 where elements are copied)."""
    y = x.copy()
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    if transposed:
        s = -s
    ia, ib = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = scale * (a * c - b * s), scale * (a * s + b * c)
    amp = np.zeros_like(x)
    amp[..., ia] = amp[..., ib] = scale * (np.abs(a) + np.abs(b))
    return y, amp


def rope_tolerance(ref: np.ndarray, amp: np.ndarray, half_step: float) -> np.ndarray:
    """The result is rounded once: half a step of its type (bf16 2^-8, fp32 2^-24).  Before that,
    cos and sin are off by the angle's error -- 2^-32 of a turn cut off and a 24-bit fraction of half a
    turn, pi 2^-25 + 2 pi 2^-32 < 2^-23.3 -- and by 2 ulp of sincospi (2^-23), times the scale's
    rounding 2^-24; two products and their sum round by 2^-24 each: under 2^-21 of |a| + |b|."""
    return half_step * np.abs(ref) + 2.0 ** -21 * amp + 1e-40


def masks_of(parents) -> list[int]:
    m = []
    for i, p in enumerate(parents):
        m.append((1 << i) | (m[p] if p >= 0 else 0))
    return m


def random_tree(rng, n: int, branch: int) -> list[int]:
    parent, kids = [-1], [0] * n
    for i in range(1, n):
        free = [j for j in range(i) if kids[j] < branch]
        p = int(rng.choice(free))
        parent.append(p)
        kids[p] += 1
    return parent


def _prob(x) -> Fraction:
    x = float(x)
    return Fraction(0) if not x > 0 else Fraction(min(x, 1.0))


def verify(tokens, parents, target, draft, u, replace: bool):
    """One sequence in exact rationals: (path, out_tokens).  target, draft [n, V] as floats."""
    n = len(tokens)
    kids: dict[int, list[int]] = {}
    for i in range(1, n):
        kids.setdefault(parents[i], []).append(i)
    num = [min(max(Fraction(float(x)), Fraction(0)), Fraction(1)) for x in u]
    cur, path, out = 0, [0], []
    while True:
        p = [_prob(x) for x in target[cur]]
        w, Z, R, nxt = list(p), Fraction(1), Fraction(1), None
        q = [_prob(x) for x in draft[cur]] if draft is not None and cur in kids else None
        for i in kids.get(cur, ()):
            x = tokens[i]
            if draft is None:
                if num[i] * Z < w[x]:
                    nxt = i
                    break
                Z, w[x] = max(Z - w[x], Fraction(0)), Fraction(0)
                continue
            if num[i] * Z * q[x] < w[x] * R:
                nxt = i
                break
            if R > 0:
                w = [max(a - Z / R * b, Fraction(0)) for a, b in zip(w, q)]
                Z = sum(w)
            if not replace:
                R -= q[x]
        if nxt is None:
            break
        cur = nxt
        path.append(cur)
        out.append(tokens[cur])
    # weights are held in units of 2^-62
    unit = 1 << 62
    if sum(w) == 0:
        w = p
    total, run, last = sum(w), Fraction(0), -1
    for x, a in enumerate(w):
        run += a
        if a * unit >= 1:
            last = x
        if run > num[0] * total:
            return path, out + [x]
    return path, out + [last]


def commit(draft_k, draft_v, path, n_path, k, v, kv_len):
    """The caches (raw bf16 bits) after the commit."""
    k, v = k.copy(), v.copy()
    for b in range(len(n_path)):
        for t in range(n_path[b]):
            x = kv_len[b] - n_path[b] + t
            k[b, :, x] = draft_k[b, :, path[b, t]]
            v[b, :, x] = draft_v[b, :, path[b, t]]
    return k, v

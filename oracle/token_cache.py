"""fp64 oracle of rotary positions and the exact token cache, written from the
formulas: numpy loops over (sequence, head), no code shared with the package.

Sources: rotary position embedding (Su et al. 2021, "RoFormer", eq. 34) with
the long-context scalings by interpolation (linear), by the base (NTK-aware),
by wavelength bands and by the YaRN ramp (Peng et al. 2023, "YaRN", eq. 23-25,
0.1 ln s + 1 for the magnitude); eviction by accumulated attention weight
(Zhang et al. 2023, "H2O", the heavy-hitter rule with recent tokens kept).
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(n, base, scaling="none", factor=1.0, original_len=8192, low=1.0, high=None):
    """(radians per position of every pair, magnitude), one pair at a time."""
    high = (32.0 if scaling == "yarn" else 4.0) if high is None else high
    out = []
    for i in range(n // 2):
        b = base
        if scaling == "ntk":
            b = base * factor ** (n / max(1.0, n - 2.0))
        f = math.pow(b, -2.0 * i / n)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            turns = original_len * f / (2 * math.pi)
            if turns <= low:
                f = f / factor
            elif turns < high:
                t = (turns - low) / (high - low)
                f = t * f + (1 - t) * f / factor
        elif scaling == "yarn":
            def at(t):
                return n * math.log(original_len / (2 * math.pi * t)) / (2 * math.log(base))
            lo = max(math.floor(at(high)), 0)
            hi = min(math.ceil(at(low)), n - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = r * f / factor + (1 - r) * f
        out.append(f)
    mag = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
    return np.array(out), mag


def rotary(x, pos, freq, mag=1.0, interleaved=False, inverse=False):
    """x [..., T, heads, d], pos [..., T]; fp64."""
    x = np.asarray(x, dtype=np.float64)
    n = len(freq)
    y = x.copy()
    ang = np.asarray(pos, dtype=np.float64)[..., None] * freq
    c, s = mag * np.cos(ang), mag * np.sin(ang)
    if inverse:
        s = -s
    for i in range(n):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        a, b = x[..., ia], x[..., ib]
        ci, si = c[..., i][..., None], s[..., i][..., None]
        y[..., ia] = a * ci - b * si
        y[..., ib] = b * ci + a * si
    return y


def attend(q, K, V, PK=None, PV=None):
    """One head group: q [G][d] over the prefix PK, PV [P][d] and own tokens
    K, V [n][d].  Returns out [G][d], lse [G], weight [n] (sum over the
    queries) and sum_i p_i |v_i| [G][d]."""
    d = q.shape[1]
    P = 0 if PK is None else len(PK)
    keys = K if P == 0 else np.concatenate((PK, K))
    vals = V if P == 0 else np.concatenate((PV, V))
    G, n = q.shape[0], len(keys)
    if n == 0:
        z = np.zeros((G, d))
        return z, np.full(G, -np.inf), np.zeros(0), z
    x = q @ keys.T / math.sqrt(d)
    m = x.max(1, keepdims=True)
    e = np.exp(x - m)
    den = e.sum(1, keepdims=True)
    p = e / den
    return p @ vals, (m + np.log(den))[:, 0], p[:, P:].sum(0), p @ np.abs(vals)


def evict(pos, weight, budget, keep_first, keep_recent):
    """Source row of every kept row, for one head's live tokens (pos, weight
    [n]): rows below keep stay where their token is kept, the kept tokens
    behind fill the gaps in order."""
    n = len(pos)
    keep = min(n, budget)
    if n == 0:
        return np.zeros(0, dtype=np.int64)
    newest = max(int(p) for p in pos)

    def rank(i):
        p = int(pos[i])
        held = p < keep_first or p > newest - keep_recent
        w = float(weight[i])
        if math.isnan(w):
            w = -math.inf
        return (0 if held else 1, 0.0 if held else -w, i)

    best = set(sorted(range(n), key=rank)[:keep])
    spare = iter(i for i in range(keep, n) if i in best)
    return np.array([j if j in best else next(spare) for j in range(keep)], dtype=np.int64)

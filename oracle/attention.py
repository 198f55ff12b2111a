"""fp64 NumPy definitions of the softmax-attention operators (include/kda_attn.h).

Written from the formulas with plain loops over sequences, heads and rows, and
sharing no code with the CUDA path.  Besides each output, :func:`prompt` and
:func:`decode` return what the tests derive tolerances from: the attention
over |v| and, per row, the largest sum of |q_i k_i| over a key's channels.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 64
E4M3_MAX = 448.0


def e4m3_values() -> np.ndarray:
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits;
    exponent and fraction all ones is NaN, there are no infinities."""
    out = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        if e == 15 and f == 7:
            x = math.nan
        elif e == 0:
            x = f * 2.0 ** -9
        else:
            x = (1 + f / 8) * 2.0 ** (e - 7)
        out[b] = -x if b & 128 else x
    return out


_VALUES = e4m3_values()
_POS = _VALUES[:127]  # 0 .. 448, increasing


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Bytes of the nearest e4m3 values, ties to the even byte, saturating; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), E4M3_MAX)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    b = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    b = np.where(np.signbit(x), b | 128, b).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7f), b)


def pow2_need(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while amax > E4M3_MAX * s:
        s *= 2.0
    return s


def _softmax(scores):
    """(weights, sum, max) of one row of scores; sum 0 for no scores."""
    if scores.size == 0:
        return scores, 0.0, -math.inf
    m = scores.max()
    w = np.exp(scores - m)
    return w, w.sum(), m


def _attend(q, k, v, scale):
    """One row: (o, lse, attention over |v|, largest scale sum |q_i k_i|)."""
    if k.shape[0] == 0:
        z = np.zeros(v.shape[1])
        return z, -math.inf, z, 0.0, np.zeros(0)
    w, total, m = _softmax(scale * (k @ q))
    p = w / total
    mag = scale * (np.abs(k) @ np.abs(q))
    return p @ v, m + math.log(total), p @ np.abs(v), float(mag.max()), p


def prompt(q, k, v, cu, scale=None):
    """q [T, Hq, d], k, v [T, Hkv, d], cu [n + 1] -> (out, lse, absout, mag)."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    absout, mag = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    for s in range(len(cu) - 1):
        for i in range(cu[s], cu[s + 1]):
            for h in range(Hq):
                out[i, h], lse[i, h], absout[i, h], mag[i, h], _ = _attend(
                    q[i, h], k[cu[s]:i + 1, h // G], v[cu[s]:i + 1, h // G], scale)
    return out, lse, absout, mag


def append(pages, scale, x, cu, start, table, transposed):
    """New page bytes and scales after appending x [T, H, d].

    pages: uint8 [N, H, 64, d], or [N, H, d, 64] when ``transposed`` (values)."""
    pages, scale = pages.copy(), scale.astype(np.float64).copy()
    if transposed:
        pages = pages.transpose(0, 1, 3, 2).copy()
    N, H = scale.shape
    for s in range(len(cu) - 1):
        n = cu[s + 1] - cu[s]
        if n == 0 or start[s] < 0:
            continue
        for c in range(start[s] // PAGE, (start[s] + n - 1) // PAGE + 1):
            lo, hi = max(start[s], c * PAGE), min(start[s] + n, (c + 1) * PAGE)
            page = table[s][c] if c < len(table[s]) else -1
            if page < 0 or page >= N:
                continue
            keep = lo - c * PAGE
            rows = x[cu[s] + lo - start[s]:cu[s] + hi - start[s]]
            for h in range(H):
                r = rows[:, h].astype(np.float64)
                fin = np.abs(r[np.isfinite(r)])
                new = pow2_need(fin.max() if fin.size else 0.0)
                if keep:
                    new = max(new, scale[page, h])
                    if new > scale[page, h]:
                        pages[page, h, :keep] = e4m3_round(_VALUES[pages[page, h, :keep]] * (scale[page, h] / new))
                pages[page, h, keep:keep + hi - lo] = e4m3_round(r / new)
                scale[page, h] = new
    if transposed:
        pages = pages.transpose(0, 1, 3, 2).copy()
    return pages, scale


def decode(q, k_pages, v_pages, k_scale, v_scale, lens, table, scale=None):
    """q [B, D, Hq, d] over the cache -> (out, lse, absout, mag, page mass [B, max_pages]).

    Positions of pages outside the cache count as unseen."""
    B, D, Hq, d = q.shape
    N, Hkv = k_scale.shape
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    width = table.shape[1]
    out, lse = np.zeros((B, D, Hq, d)), np.full((B, D, Hq), -math.inf)
    absout, mag = np.zeros((B, D, Hq, d)), np.zeros((B, D, Hq))
    mass = np.zeros((B, width))
    for n in range(B):
        length = min(max(int(lens[n]), 0), width * PAGE)
        ids = [int(x) for x in table[n, :-(-length // PAGE)]]
        good = np.repeat([0 <= x < N for x in ids], PAGE)[:length] if ids else np.zeros(0, bool)
        safe = [x if 0 <= x < N else 0 for x in ids]
        for h in range(Hkv):
            if not ids:
                continue
            k = np.concatenate([_VALUES[k_pages[x, h]] * k_scale[x, h] for x in safe])[:length]
            v = np.concatenate([_VALUES[v_pages[x, h]].T * v_scale[x, h] for x in safe])[:length]
            for t in range(D):
                end = max(0, length - D + 1 + t)
                at = np.nonzero(good[:end])[0]
                for g in range(h * G, (h + 1) * G):
                    o, e, a, m, p = _attend(q[n, t, g], k[at], v[at], scale)
                    out[n, t, g], lse[n, t, g], absout[n, t, g], mag[n, t, g] = o, e, a, m
                    if at.size:
                        np.add.at(mass[n], at // PAGE, p)
    return out, lse, absout, mag, mass


def evict(lens, table, weight, budget, sink, recent):
    """(lens, table, weight, freed, count) after dropping the lightest pages."""
    B, width = table.shape
    lens, new_t, new_w = lens.copy(), np.full_like(table, -1), np.zeros_like(weight)
    freed, count = np.full_like(table, -1), np.zeros(B, np.int32)
    for n in range(B):
        P = max(0, -(-int(lens[n]) // PAGE))
        gone = set()
        if P <= width and P > budget:
            def key(c):
                w = float(weight[n, c])
                return (-math.inf if math.isnan(w) else w, 0 if math.isnan(w) else 1, -c)
            gone = set(sorted(range(sink, P - recent), key=key)[:P - budget])
        kept = [c for c in range(width) if c not in gone]
        new_t[n, :len(kept)] = table[n, kept]
        new_w[n, :len(kept)] = weight[n, kept]
        out = sorted(gone)
        freed[n, :len(out)] = table[n, out]
        count[n] = len(out)
        lens[n] -= PAGE * len(out)
    return lens, new_t, new_w, freed, count

"""Plain oracle of the paged 8-bit cache (numpy, float64 where a value is computed).

Written from the definitions in include/vq.h, one page, token or query at a time;
nothing here is shared with the CUDA side. A cache is a dict: "k", "v" uint8
[pages][H][64][D], "k_scale", "v_scale" float32 [pages][H], "pos" int32 and
"weight" float32 [pages][H][64] (or None), "fmt" "int8" or "e4m3".
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

PAGE = 64
CUT = float(2.0 ** 126)


def e4m3_table():
    """The value of each of the 256 e4m3 codes (NaN for the two NaN codes)."""
    v = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7)
        if b & 127 == 127:
            x = np.nan
        v[b] = -x if b & 128 else x
    return v


_E4M3 = e4m3_table()
_E4M3_POS = _E4M3[:127]  # 0 .. 448, increasing


def code_values(raw, fmt):
    """float64 values of code bytes."""
    raw = np.asarray(raw, dtype=np.uint8)
    return raw.view(np.int8).astype(np.float64) if fmt == "int8" else _E4M3[raw]


def encode(x, fmt):
    """Code bytes of the nearest codes to x (float64, exact inputs), ties to even."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    mag = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_E4M3_POS, mag, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = mag - _E4M3_POS[lo], _E4M3_POS[hi] - mag
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def fresh_scale(amax, fmt):
    """Scale of a page first written with largest magnitude amax (an exact float32)."""
    if amax == 0:
        return np.float32(0)
    if fmt == "int8":
        return max(np.float32(amax) / np.float32(127), np.float32(2.0 ** -126))
    e = -126
    while Fraction(float(amax)) > 448 * Fraction(2) ** e:
        e += 1
    return np.float32(2.0 ** e)


def grown(scale, amax, fmt):
    """(new scale, k): the smallest power of two that makes amax fit a page of this scale."""
    k, s, a = 0, Fraction(float(scale)), Fraction(float(amax))
    while (a * 2 >= 255 * s * 2 ** k) if fmt == "int8" else (a > 448 * s * 2 ** k):
        k += 1
    return np.float32(float(s * 2 ** k)), k


def quotient_codes(x, scale, fmt):
    """Codes of the real quotients x / scale."""
    if scale == 0:
        return np.zeros(np.shape(x), np.uint8)
    x = np.asarray(x, dtype=np.float64)
    # float64: x has 24 bits and so has scale; a quotient that is not half-way between two codes is at
    # least 2^-25 of itself away, so rounding it to 53 bits cannot put it there
    return encode(x / np.float64(scale), fmt)


def append(c, table, start, counts, k, v, pos=None):
    """k, v float32 [B][H][n][D]; changes the cache in place."""
    B, H, n, D = k.shape
    for b in range(B):
        lo_t, hi_t = int(start[b]), int(start[b]) + int(counts[b])
        for p in range(lo_t // PAGE, (hi_t - 1) // PAGE + 1 if hi_t > lo_t else lo_t // PAGE):
            page = int(table[b][p])
            s0, s1 = max(lo_t - p * PAGE, 0), min(hi_t - p * PAGE, PAGE)
            for h in range(H):
                for name, x in (("k", k), ("v", v)):
                    new = np.asarray(x[b, h, p * PAGE + s0 - lo_t:p * PAGE + s1 - lo_t], dtype=np.float64)
                    new = np.clip(np.where(np.isnan(new), 0.0, new), -CUT, CUT)
                    amax = np.abs(new).max()
                    old = c[name + "_scale"][page, h] if s0 > 0 else np.float32(0)
                    if old > 0:
                        scale, g = grown(old, amax, c["fmt"])
                        if g:
                            was = code_values(c[name][page, h, :s0], c["fmt"])
                            c[name][page, h, :s0] = encode(was * 2.0 ** -g, c["fmt"])
                    else:
                        scale = fresh_scale(amax, c["fmt"])
                    c[name + "_scale"][page, h] = scale
                    c[name][page, h, s0:s1] = quotient_codes(new, scale, c["fmt"])
                at = np.arange(s0, s1)
                if c["pos"] is not None:
                    first = lo_t if pos is None else int(pos[b])
                    c["pos"][page, h, s0:s1] = first + p * PAGE + at - lo_t
                if c["weight"] is not None:
                    c["weight"][page, h, s0:s1] = 0.0


def read(c, table, b, h, begin, end):
    """float32 values of K and V of tokens begin .. end - 1."""
    out = []
    for name in ("k", "v"):
        rows = []
        for t in range(begin, end):
            page = int(table[b][t // PAGE])
            rows.append(code_values(c[name][page, h, t % PAGE], c["fmt"]).astype(np.float32)
                        * c[name + "_scale"][page, h])
        out.append(np.array(rows, dtype=np.float32).reshape(end - begin, c[name].shape[-1]))
    return out


def per_slot(c, name, table, b, h, n):
    return np.array([c[name][int(table[b][t // PAGE]), h, t % PAGE] for t in range(n)])


def scores(c, table, b, h, hq, length, q, sigma, *, q_len, q_pos=None, prefix=0, first=None, slope=0.0, cap=0.0,
           causal=False):
    """z [q_len][length] of one query head's queries q [q_len][D], -inf where unseen, and a bound of its float32 error."""
    k = read(c, table, b, h, 0, length)[0].astype(np.float64)
    raw = sigma * (q @ k.T)
    err = sigma * (np.abs(q) @ np.abs(k).T) * (q.shape[1] + 16) * 2.0 ** -24 + np.abs(raw) * 2.0 ** -22
    z = raw
    if cap > 0:
        z = cap * np.tanh(raw / cap)
        # small scores by a polynomial (eight float32 roundings of the score), larger ones by exponentials (of the cap)
        err = err + np.where(np.abs(raw) <= 0.2499 * cap, np.abs(raw), cap) * 2.0 ** -21
    slot = np.arange(length)
    kp = per_slot(c, "pos", table, b, h, length) if c["pos"] is not None else slot
    own = length - q_len + np.arange(q_len)
    qp = own if q_pos is None else q_pos + np.arange(q_len)
    bias = slope * np.abs(qp[:, None] - kp[None])
    z = z - bias
    err = err + (np.abs(bias) + np.abs(z)) * 2.0 ** -22
    see = np.ones((q_len, length), bool)
    if causal:
        see = (slot[None] <= own[:, None]) | (kp[None] < prefix)
    if first is not None:
        see &= kp[None] >= np.asarray(first)[:q_len, None]
    return np.where(see, z, -np.inf), err


def attention(z, v):
    """(out, lse, weights) of scores z [n][L] over values v [L][D]."""
    n, D = z.shape[0], v.shape[1]
    out, lse, w = np.zeros((n, D)), np.full(n, -np.inf), np.zeros(z.shape)
    for i in range(n):
        if z.shape[1] and np.isfinite(z[i]).any():
            m = z[i].max()
            e = np.exp(z[i] - m)
            lse[i] = m + np.log(e.sum())
            w[i] = e / e.sum()
            out[i] = w[i] @ v
    return out, lse, w


def keep_slots(w, length, keep, sinks, recent):
    """Slots that an eviction keeps of one head's weights, ascending."""
    if length <= keep:
        return list(range(length))
    rest = range(sinks, length - recent)
    key = [(-np.inf if np.isnan(w[j]) else float(w[j])) for j in range(length)]
    best = sorted(rest, key=lambda j: (-key[j], j))[:keep - sinks - recent]
    return sorted(list(range(sinks)) + best + list(range(length - recent, length)))


def evict(c, table, lens, to, to_table, keep, sinks, recent):
    """Fills `to` in place; returns (kept [B][H][keep], new lengths)."""
    B, H = len(lens), c["k"].shape[1]
    kept = np.full((B, H, keep), -1, np.int32)
    for b in range(B):
        L = int(lens[b])
        for h in range(H):
            w = per_slot(c, "weight", table, b, h, L)
            at = keep_slots(w, L, keep, sinks, recent)
            kept[b, h, :len(at)] = at
            for p in range(0, len(at), PAGE):
                part = at[p:p + PAGE]
                dst = int(to_table[b][p // PAGE])
                src = [int(table[b][j // PAGE]) for j in part]
                for name in ("k", "v"):
                    scale = np.array([c[name + "_scale"][s, h] for s in src])
                    top = scale.max()
                    to[name + "_scale"][dst, h] = top
                    for i, (s, j) in enumerate(zip(src, part)):
                        raw = c[name][s, h, j % PAGE]
                        if scale[i] != top:
                            raw = encode(code_values(raw, c["fmt"]) * np.float64(scale[i]) / np.float64(top), c["fmt"])
                        to[name][dst, h, i] = raw
                for i, (s, j) in enumerate(zip(src, part)):
                    if to["pos"] is not None:
                        to["pos"][dst, h, i] = c["pos"][s, h, j % PAGE] if c["pos"] is not None else j
                    if to["weight"] is not None:
                        to["weight"][dst, h, i] = c["weight"][s, h, j % PAGE]
    return kept, np.minimum(np.asarray(lens), keep)

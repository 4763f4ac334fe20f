"""Plain 64-bit forms of the 8-bit cache's operators (numpy, float64), and the
tolerances their GPU counterparts are held to.

Cache layout: k, v e4m3 bytes [NP][Hkv][P][D]; scales E8M0 bytes
[NP][Hkv][P/16][2] (K, V).
"""
from __future__ import annotations

import numpy as np

E_MIN, E_MAX = -60, 40

# value of every e4m3 byte (the format has no infinity; 0x7f and 0xff are NaN)
_B = np.arange(256)
_EXP, _MAN = (_B >> 3) & 15, _B & 7
VALUES = np.where(_EXP == 0, _MAN * 2.0 ** -9, (8 + _MAN) * 2.0 ** (_EXP - 10.0))
VALUES = np.where(_B & 128, -VALUES, VALUES)
VALUES[0x7F] = VALUES[0xFF] = np.nan


def encode(x):
    """float64 -> e4m3 bytes: to nearest, ties to even, beyond 448 to 448; not
    finite -> NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(np.where(np.isfinite(a), a, 1.0))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    r = np.rint(a / step) * step  # may reach the next binade: still a value
    pos = VALUES[:0x7F]           # ascending
    idx = np.searchsorted(pos, np.where(np.isfinite(r), r, 0.0))
    assert np.all((pos[np.minimum(idx, 0x7E)] == r) | ~np.isfinite(x))
    out = idx.astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isfinite(x), out, np.uint8(0x7F)).astype(np.uint8)


def need_exp(a):
    """Smallest e with a <= 448 * 2^e, clamped; a >= 0."""
    if a == 0:
        return E_MIN
    e = E_MIN
    while e < E_MAX and a > 448.0 * 2.0 ** e:
        e += 1
    return e


def runs(positions, seq_ids):
    """(first token, tokens) of every run: consecutive tokens of one sequence at
    consecutive positions of one block; skipped tokens belong to none."""
    out = []
    n = len(positions)
    i = 0
    while i < n:
        if positions[i] < 0:
            i += 1
            continue
        j = i + 1
        while (j < n and seq_ids[j] == seq_ids[i] and positions[j] == positions[j - 1] + 1
               and positions[j] % 16):
            j += 1
        out.append((i, j - i))
        i = j
    return out


def append(k, v, scales, k_new, v_new, table, positions, seq_ids):
    """In place on uint8 arrays; k_new, v_new float64 [tokens][Hkv][D]."""
    P = k.shape[2]
    for i, n in runs(positions, seq_ids):
        page = table[seq_ids[i]][positions[i] // P]
        lo = positions[i] % P
        blk, first = lo // 16, lo // 16 * 16
        for side, (x, pool) in enumerate(((k_new, k), (v_new, v))):
            for h in range(k.shape[1]):
                y = x[i:i + n, h]
                fin = np.abs(y[np.isfinite(y)])
                e = need_exp(fin.max() if fin.size else 0.0)
                if lo > first:
                    old = int(np.clip(int(scales[page, h, blk, side]) - 127, E_MIN, E_MAX))
                    if e > old:
                        rows = pool[page, h, first:lo]
                        vals = VALUES[rows]
                        again = encode(vals * 2.0 ** (old - e))
                        pool[page, h, first:lo] = np.where(np.isnan(vals), rows | 0x7F, again)
                    e = max(e, old)
                pool[page, h, lo:lo + n] = encode(y * 2.0 ** -e)
                scales[page, h, blk, side] = e + 127


def norm_rope(x, weight, positions, theta, eps):
    """x float64 [tokens][heads][D]."""
    D = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    if theta:
        inv = theta ** (-np.arange(0, D, 2) / D)
        a = (np.asarray(positions, dtype=np.float64)[:, None] * inv)[:, None, :]
        c, s = np.cos(a), np.sin(a)
        p, q = x[..., :D // 2], x[..., D // 2:]
        x = np.concatenate([p * c - q * s, q * c + p * s], -1)
    return x


def dense(pool, scales, side, row, n):
    """The first n tokens of a table row, [Hkv][n][D] in float64."""
    P = pool.shape[2]
    pages = row[:(n + P - 1) // P]
    e = scales[pages][..., side].astype(np.float64) - 127
    x = VALUES[pool[pages]] * np.repeat(2.0 ** e, 16, axis=2)[..., None]
    return np.moveaxis(x, 0, 1).reshape(pool.shape[1], -1, pool.shape[3])[:, :n]


def attention(q, k, v, scales, table, lens, scale):
    """q float64 [B][Q][Hq][D].  Returns out and, per output, the bound's parts:
    a (the same weighted mean of |v|), and vmax (largest |v| the row sees)."""
    B, Q, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mean, vmax = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        kk, vv = dense(k, scales, 0, table[b], n), dense(v, scales, 1, table[b], n)
        for j in range(Q):
            m = n - Q + j + 1  # tokens query j sees
            if m <= 0:
                continue
            for h in range(Hq):
                s = kk[h // G, :m] @ q[b, j, h] * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[b, j, h] = w @ vv[h // G, :m]
                mean[b, j, h] = w @ np.abs(vv[h // G, :m])
                vmax[b, j, h] = np.abs(vv[h // G, :m]).max()
    return out, mean, vmax


def attention_bound(ref, mean, vmax, lens, half_step, score_err):
    """How far a computed output may be from the exact one.

    half_step: the output's rounding, relative to the value (bf16 2^-8, fp16
    2^-11).  The weights are rounded to fp16, 2^-11 each, which moves the
    weighted sum by at most 2^-11 of the weighted mean of |v|; a weight below
    fp16's normal range (2^-14; the row's largest is at least 1) loses at most
    2^-25, on at most n tokens.  Scores off by score_err (absolute, natural
    units) move each weight, and the sum of weights, by that much relative.
    fp32 sums: n * 2^-24 on either side of the division, and 2^-20 for the
    exponentials and the division."""
    n = np.maximum(np.asarray(lens, dtype=np.float64), 1).reshape(-1, 1, 1, 1)
    rel = 2.0 ** -11 + 2 * score_err + 2 * n * 2.0 ** -24 + 2.0 ** -20
    d = mean * rel + vmax[..., None] * n * 2.0 ** -25 * 2
    return d + half_step * (np.abs(ref) + d) + 1e-30

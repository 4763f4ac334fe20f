"""How far an output of the 8-bit cache's attention may be from the exact one, row by
row, and caches made to show where it is not.

The bound uses each token's own value and its own weight: a large value somewhere in
the cache widens no row that gives it no weight.  With s the exact scores, w_t =
e^(s_t) over its sum:

* scores.  A product's fp32 accumulator takes D exact products; the tensor core may
  cut each of the terms that it aligns to the largest one instead of rounding it:
  2 D 2^-23 of the sum of magnitudes.  The exponent x = s log2 e + e_v and x - m are
  rounded a few times: 2^-22 of their size.  Either moves a weight by as much,
  relative, and the sum of the weights by their mean.
* weights.  16 bits with 11 of fraction, 2^-11 of w_t |v_t|; a weight below 2^-14 of the
  row's sum loses at most 2^-25 of it, never more than itself, nor more than 2^-32 of
  the largest w_t 2^e_v in its own V scale 2^e_v.
* sums of n terms, cut like those of the scores: 2 n 2^-23; 2^-18 for the exponentials,
  the merges and the division.
* the output's rounding, half a step of it (and half of fp16's smallest subnormal).
"""
from __future__ import annotations

import numpy as np

import kv8_ref as ref

HALF = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


def attention(q, k, v, scales, table, lens, scale, dtype):
    """q float64 [B][Q][Hq][D], the cache as kv8_ref has it -> (exact output, bound), both
    of q's shape; dtype: the outputs' ("bfloat16" or "float16")."""
    B, Q, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    out, lim = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        kk, vv = (ref.dense(p, scales, x, table[b], n) for x, p in enumerate((k, v)))
        ev = np.clip(scales[table[b][:-(-n // k.shape[2])]][..., 1].astype(int) - 127,
                     ref.E_MIN, ref.E_MAX)               # [pages][H][blocks]
        ev = np.repeat(np.moveaxis(ev, 1, 0).reshape(H, -1), 16, axis=1)[:, :n]
        see = np.arange(n) <= (n - Q + np.arange(Q))[:, None]  # [Q][n]
        see = np.repeat(see, G, axis=0)
        any_ = see.any(1)
        for h in range(H):
            rows = q[b, :, h * G:(h + 1) * G].reshape(Q * G, D)
            s = rows @ kk[h].T * scale
            size = np.abs(rows) @ np.abs(kk[h]).T * abs(scale)
            s = np.where(see, s, -np.inf)
            m = np.where(any_, s.max(1, initial=-np.inf), 0.0)
            w = np.exp(s - m[:, None])
            w /= np.maximum(w.sum(1, keepdims=True), 1e-300)
            far = (w * 2.0 ** ev[h]).max(1, keepdims=True) * 2.0 ** (-32.0 - ev[h])
            lost = np.minimum(np.minimum(w, 2.0 ** -25), far)
            d_s = np.where(see, size * 2 * D * 2.0 ** -23 + (np.abs(s) * 1.4427 + np.abs(ev[h]).max())
                           * 2.0 ** -22, 0.0)
            assert (w * d_s).sum(1).max() < 4e-3, "scores too large for a bound of a percent"
            rel = d_s + (w * d_s).sum(1, keepdims=True) + 2.0 ** -11 + 2 * n * 2.0 ** -23 + 2.0 ** -18
            a = np.abs(vv[h])
            o = w @ vv[h]
            d = (rel * w + lost) @ a
            d += HALF[dtype] * (np.abs(o) + d) + (2.0 ** -25 if dtype == "float16" else 1e-38)
            out[b, :, h * G:(h + 1) * G] = o.reshape(Q, G, D)
            lim[b, :, h * G:(h + 1) * G] = d.reshape(Q, G, D)
    return out, lim


def check(c, q, out, scale):
    """out [B][Q][Hq][D] (torch) against the exact attention over c (a Cache)."""
    want, lim = attention(q.double().cpu().numpy(), c.k, c.v, c.scales, c.table, c.lens, scale,
                          str(q.dtype).split(".")[1])
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > lim
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[0],
                           float((np.abs(got - want) / lim).max()))


def fill(c, k, v):
    """c's cache from dense values: k, v [B] lists of [tokens][Hkv][D] float64."""
    for b, n in enumerate(c.lens):
        for side, (x, pool) in enumerate(((k[b], c.k), (v[b], c.v))):
            y = np.zeros((-(-int(n) // 16) * 16, *x.shape[1:]))
            y[:n] = x[:n]
            y = y.reshape(-1, 16, *x.shape[1:])         # [blocks][16][Hkv][D]
            f, e = np.frexp(np.abs(y).max((1, 3)) / 448)  # f 2^e, f in [0.5, 1)
            e = np.where(f == 0.5, e - 1, e)
            e = np.where(f == 0, ref.E_MIN, np.clip(e, ref.E_MIN, ref.E_MAX))
            by = ref.encode(y * 2.0 ** -e[:, None, :, None])
            for i in range(len(y)):
                page, at = c.table[b][i * 16 // c.P], i * 16 % c.P
                pool[page, :, at:at + 16] = by[i].transpose(1, 0, 2)
                c.scales[page, :, at // 16, side] = e[i] + 127
    return c


def edges(c, q, Q):
    """Rows that show which tokens they saw: the keys of each sequence's last Q + 1
    tokens get weights that no row's result can hide, and their values a size of their own.
    q (float64 [B][Q][Hq][D], in place): element 0 is 3 in every row.  Returns c."""
    q[..., 0] = 3.0
    k, v = [], []
    for n in c.lens:
        n = int(n)
        x = c.rng.standard_normal((2, n, c.Hkv, c.D))
        x[0, :, :, 0] = 0.0
        lo = max(0, n - Q - 1)
        # the same weight for every row, of the last ones together about that of the rest
        x[0, lo:] = 0.0
        x[0, lo:, :, 0] = np.log(max(1.0, 2.0 * n / (n - lo + 1.0))) / 3.0 * c.D ** 0.5
        x[1, lo:] += 3.0 * np.sign(x[1, lo:])
        k.append(x[0])
        v.append(x[1])
    return fill(c, k, v)

"""Plain forms in 64 bits of the calls that serve with selected pages, on the CPU,
and the bounds that the GPU's results are held to."""
from __future__ import annotations

import math

import numpy as np
import torch

BAD_PAGE, BAD_LEN, NO_PAGES = 0x1, 0x2, 0x20
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}  # half the smallest step


def rounded(ref, err, dtype):
    """What a value within err of ref may be off by after its rounding to dtype."""
    return err + HALF[dtype] * (ref.abs() + err) + TINY[dtype]


def close(got, ref, bound, what=""):
    got = got.double().cpu()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN in other places"
    bad = ((got - ref).abs() > bound) & ~ref.isnan()
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[i].item()!r} for {ref[i].item()!r}, bound "
                             f"{bound[i].item():.3g}")


def tables(cached, new, free, begin, table, page, num_pages, n_tokens):
    """-> (table, lens, starts, positions, seq_ids, slots, free_end, status)."""
    table = [list(r) for r in table]
    cols = len(table[0]) if table else 0
    pos, seq, slots = ([-1] * n_tokens for _ in range(3))
    lens, starts, status = [], [0], 0
    avail = len(free) - begin
    if begin < 0 or avail < 0:
        avail, status = 0, NO_PAGES
    asked = taken = row = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        ok = c >= 0 and n >= 0
        c, n = max(c, 0), max(n, 0)
        first = row
        row += n
        if not ok or c + n > min(cols * page, 2 ** 31 - 1) or row > n_tokens:
            status |= BAD_LEN
            ok = False
        else:
            have, need = -(-c // page), -(-(c + n) // page) - -(-c // page)
            if need and asked + need > avail:
                status |= NO_PAGES
                ok = False
            at = begin + asked
            asked += need
            if ok and need:
                table[b][have:have + need] = free[at:at + need]
                taken = asked
        for i in range(first, min(row, n_tokens)):
            seq[i] = b
            if ok:
                p = c + i - first
                pos[i] = p
                pg = table[b][p // page]
                if 0 <= pg < num_pages:
                    slots[i] = pg * page + p % page
                else:
                    status |= BAD_PAGE
        lens.append(c + n if ok else c)
        starts.append(min(row, n_tokens))
    return table, lens, starts, pos, seq, slots, begin + taken, status


def frequencies(rdim, theta, scaling="none", factor=1.0, low=1.0, high=4.0, context=8192.0):
    i = np.arange(rdim // 2, dtype=np.float64)
    f = theta ** (-2 * i / rdim)
    if scaling == "linear":
        return f / factor
    if scaling == "turns":
        keep = np.clip((context * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return keep * f + (1 - keep) * f / factor
    if scaling == "index":
        def at(n):
            return rdim / (2 * math.log(theta)) * math.log(context / (2 * math.pi * n))
        lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rdim - 1)
        keep = 1 - np.clip((i - lo) / (max(hi, lo + 0.001) - lo), 0, 1)
        return keep * f + (1 - keep) * f / factor
    return f


def turned(x, pos, freq, interleaved, magnitude=1.0, weight=None, eps=0.0):
    """x [tokens, heads, D] (any dtype) -> (exact rows, a bound on the error of fp32
    arithmetic on them), both [tokens, heads, D] in 64 bits."""
    x = x.double().cpu()
    D = x.shape[-1]
    scale = torch.ones(())
    if weight is not None:
        scale = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double().cpu()
    x = x * scale
    r = 2 * len(freq)
    a = pos.double().cpu()[:, None, None] * torch.from_numpy(np.asarray(freq))
    c, s = a.cos() * magnitude, a.sin() * magnitude
    one, two = ((slice(0, r, 2), slice(1, r, 2)) if interleaved
                else (slice(0, r // 2), slice(r // 2, r)))
    y = x.clone()
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    # cos and sin: two units in the last place of a value up to 1, and the angle's own
    # rounding (2^-25 of half a turn, pi 2^-25): 2^-21 in all; the norm: D roundings of its
    # sum at worst (only positive terms: 2^-24 each relative, halved by the root), the
    # quotient and two products; three roundings of products and sum
    size = x.abs()
    both = size.clone()
    both[..., one] = both[..., two] = (size[..., one] + size[..., two]) * magnitude
    rel = (D / 2 + 4) * 2.0 ** -24 if weight is not None else 0.0
    err = both * (2.0 ** -21 + 3 * 2.0 ** -24 + rel)
    if weight is None:
        err[..., r:] = 0.0
    return y, err


def page_bounds(k_pool, slots, bounds, page):
    """k_pool [NP, Hkv, P, D], slots a list -> the new bounds."""
    out = bounds.clone()
    for i, s in enumerate(slots):
        if s < 0:
            continue
        if i + 1 < len(slots) and slots[i + 1] == s + 1 and (s + 1) % page:
            continue
        rows = k_pool[s // page, :, :s % page + 1]
        out[s // page, :, 0], out[s // page, :, 1] = rows.amin(1), rows.amax(1)
    return out


def scores(q, bounds, ids, num_pages):
    """q [G, D], bounds [NP, 2, D] of one head, ids: page ids -> scores in 64 bits."""
    q = q.double().cpu()
    up = torch.where(torch.signbit(q), torch.zeros_like(q), q)
    down = torch.where(torch.signbit(q), q, torch.zeros_like(q))
    out = []
    for p in ids:
        if not 0 <= p < num_pages:
            out.append(-math.inf)
            continue
        lo, hi = bounds[p, 0].double(), bounds[p, 1].double()
        x = (up * hi + down * lo).sum(-1)
        out.append(math.nan if x.isnan().any() else x.max().item())
    return out


def select(q, bounds, table, lens, page, max_pages, first, last):
    """-> ([B][Hkv] lists of max_pages indexes, status)."""
    bounds = bounds.cpu()
    NP, Hkv = bounds.shape[:2]
    G = q.shape[1] // Hkv
    cols = len(table[0])
    res, status = [], 0
    for b, n_tok in enumerate(lens):
        if n_tok < 0 or n_tok > cols * page:
            status |= BAD_LEN
            n_tok = min(max(n_tok, 0), cols * page)
        n = -(-n_tok // page)
        row = []
        for h in range(Hkv):
            if n <= max_pages:
                take = list(range(n))
            else:
                if max_pages > first + last and any(not 0 <= p < NP for p in table[b][:n]):
                    status |= BAD_PAGE  # (looked at only where there is something to choose)
                sc = scores(q[b, h * G:h * G + G], bounds[:, h], table[b][first:n - last], NP)
                order = sorted(range(len(sc)),
                               key=lambda i: (0 if math.isnan(sc[i]) else 1,
                                              0 if math.isnan(sc[i]) else -sc[i], i))
                want = max_pages - first - last
                take = sorted([i + first for i in order[:want]] + list(range(first)) +
                              list(range(n - last, n)))
            row.append(take + [-1] * (max_pages - len(take)))
        res.append(row)
    return res, status


def attend(q, k_pool, v_pool, table, lens, selected, scale):
    """-> (exact outputs, a bound on them) [B, Hq, D] in 64 bits."""
    dtype = q.dtype
    q, k_pool, v_pool = q.cpu().double(), k_pool.cpu(), v_pool.cpu()
    B, Hq, D = q.shape
    NP, Hkv, P, _ = k_pool.shape
    G = Hq // Hkv
    cols = len(table[0])
    out, bound = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D,
                                                                       dtype=torch.float64)
    for b in range(B):
        n_tok = min(max(int(lens[b]), 0), cols * P)
        for h in range(Hkv):
            ks, vs = [], []
            before = None
            for j in selected[b][h]:
                usable = 0 <= j < -(-n_tok // P) and (before is None or j > before)
                before = j
                if not usable or not 0 <= table[b][j] < NP:
                    continue
                m = min(P, n_tok - j * P)
                ks.append(k_pool[table[b][j], h, :m])
                vs.append(v_pool[table[b][j], h, :m])
            if not ks:
                bound[b, h * G:h * G + G] = TINY[dtype]
                continue
            k, v = torch.cat(ks).double(), torch.cat(vs).double()
            rows = slice(h * G, h * G + G)
            x = q[b, rows] @ k.T * scale
            w = torch.softmax(x, -1)
            o = w @ v
            # a score: D products summed in fp32 (2^-24 of the sum so far each, cut rather
            # than rounded: twice that), the scale and the difference to the maximum
            s_err = (q[b, rows].abs() @ k.abs().T * abs(scale)).amax(-1) * (D + 4) * 2.0 ** -23
            # a weight: both scores of its difference, exp2 and its sum, the running factor
            # of each of the chunks; its rounding to 11 (fp16) or 16 (bf16, two parts) bits
            n = k.shape[0]
            w_err = 2 * s_err + (n / 16 + 8) * 2.0 ** -22 + (
                2.0 ** -11 if dtype == torch.float16 else 2.0 ** -15)
            e = (w @ v.abs()) * w_err[:, None]
            if dtype == torch.float16:  # weights below 2^-14 of the largest: absolute steps
                e = e + n * 2.0 ** -25 * v.abs().amax(0) * w.amax(-1, keepdim=True)
            out[b, rows], bound[b, rows] = o, rounded(o, e, dtype)
    return out, bound

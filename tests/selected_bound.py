"""A bound on every element of the attention over selected pages, for both types with P in
two pieces: what each step of the kernel's arithmetic may cost, and no more."""
import math

import torch

from selected_ref import TINY, rounded

# P's two pieces keep so much of a weight, relatively, and of the largest weight.
# bf16: 8 bits, cut, and 8 of the rest, rounded: 2^-7 2^-9; fp16: 2^-10 2^-12, and at the
# range's lower end a step of 2^-24 under a largest weight of 2^15.
PIECES = {torch.bfloat16: (2.0 ** -16, 0.0), torch.float16: (2.0 ** -22, 2.0 ** -39)}


def steps(lists, page):
    """The most chunks of 16 tokens that one warp takes: they are dealt out by their places
    in the list, over 6 or 8 warps or a multiple of 8."""
    per = page // 16
    at = [e * per + i for e, j in enumerate(lists) if j >= 0 for i in range(per)]
    return max([sum(c % w == r for c in at) for w in (6, 8) for r in range(w)], default=0)


def attend(q, k_pool, v_pool, table, lens, selected, scale):
    """-> (exact outputs, bounds) [B, Hq, D] in 64 bits; lists of ascending entries, -1 behind."""
    dtype = q.dtype
    rel, low = PIECES[dtype]
    q, k_pool, v_pool = q.cpu().double(), k_pool.cpu().double(), v_pool.cpu().double()
    B, Hq, D = q.shape
    _, Hkv, P, _ = k_pool.shape
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    bound = torch.full_like(out, TINY[dtype])
    for b in range(B):
        for h in range(Hkv):
            ids = [j for j in selected[b][h] if j >= 0]
            if not ids:
                continue
            k, v = (torch.cat([x[table[b][j], h, :min(P, lens[b] - j * P)] for j in ids])
                    for x in (k_pool, v_pool))
            rows = slice(h * G, h * G + G)
            x = q[b, rows] @ k.T * scale
            w = torch.softmax(x, -1)
            # a score: the products that are not 0, each added into a sum in fp32 (cut:
            # 2^-23 of it); the scale, its own rounding and the difference to the maximum.
            # e^s_err - 1 <= 2 s_err twice: its own and the maximum's weight
            terms = (q[b, rows] != 0).sum(-1)
            size = (q[b, rows].abs() @ k.abs().T * abs(scale)).amax(-1)
            s_err = size * ((terms > 1) * terms * 2.0 ** -23 + 4 * 2.0 ** -24)
            # exp2 (2^-22) and the pieces; a step: two products of 16 terms and the sum so
            # far, each term cut at 2^-24 of the largest, the factor of a new maximum and its
            # product, the same for the sum of the weights; the merge of up to 8 warps and
            # 8 CTAs; the quotient
            w_err = 4 * s_err + 2.0 ** -22 + rel + steps(selected[b][h], P) * (
                34 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -23) + 2.0 ** -20 + 2.0 ** -20 + 2.0 ** -22
            o = w @ v
            e = (w @ v.abs()) * w_err[:, None] + w.amax(-1, keepdim=True) * low * v.abs().sum(0)
            out[b, rows], bound[b, rows] = o, rounded(o, e, dtype)
    return out, bound


def cancelling(dtype, seed, tokens=96, d=64):
    """A request of one KV head and 4 query heads whose outputs cancel, so that their own
    rounding hides nothing: q has one element, which makes the scores exact, and the last
    token's values take away what the others add up to for the first head.
    -> q, k_pool, v_pool, table, lens, lists, scale."""
    gen = torch.Generator().manual_seed(seed)
    pages = tokens // 16
    q = torch.zeros(1, 4, d, dtype=dtype)
    q[0, :, 3] = torch.tensor([1.0, -1.0, 0.5, 2.0])
    k = torch.randn(pages, 1, 16, d, generator=gen).to(dtype)
    v = torch.randn(pages, 1, 16, d, generator=gen).to(dtype)
    k[-1, 0, -1, 3] = 2.0
    x = q.double()[0] @ k.double().reshape(tokens, d).T
    w = torch.softmax(x, -1)[0]
    v[-1, 0, -1] = -(w[:-1] @ v.double().reshape(tokens, d)[:-1] / w[-1]).to(dtype)
    return q, k, v, [list(range(pages))], [tokens], [[list(range(pages))]], 1.0


def tail(dtype, drop, tokens=32768, d=64, page=256):
    """A token without values that outweighs each of the others, of values 1024, 2^drop
    times: the output is 1024 n 2^-drop / (1 + n 2^-drop)."""
    pages = tokens // page
    q = torch.zeros(1, 2, d, dtype=dtype)
    q[0, :, 0] = 1.0
    k = torch.zeros(pages, 1, page, d, dtype=dtype)
    v = torch.full((pages, 1, page, d), 1024.0, dtype=dtype)
    k[0, 0, 5, 0] = drop
    v[0, 0, 5] = 0.0
    return q, k, v, [list(range(pages))], [tokens], [[list(range(pages))]], math.log(2.0)

"""The 8-bit paged cache: what is measured.

Operators: the append of new keys and values to a cache held in e4m3 with one
power-of-two scale for each block of 16 tokens, KV head and side (with the
norms and the rotation of q and k on the way), decode attention of one query
token over that cache, of several causal query tokens, and the serving step
(append, then decode).

A block's scale is 2^e, stored as E8M0 in scales[page][head][block][side]
(side 0: K, 1: V).  A run of new tokens of one block needs the smallest e with
max|x| <= 448 * 2^e, at least -60 and at most 40; a run that starts at the
block's first slot sets the scale to that, another one takes the larger of that
and the block's old scale, and rounds the block's earlier rows to a larger scale.
"""
import math

import torch

own = False

BLOCK = 16
E_MIN, E_MAX = -60, 40
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, batch, lo, hi, hq, hkv, d, page, dtype, queries=1, rope=0.0, norm=False,
          empty=0):
    c = dict(op=op, batch=batch, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype,
             queries=queries, rope=rope, norm=norm, empty=empty)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one sequence, no rotation: the smallest write
        _case("append_token", "append", 1, 1, 1, 4, 2, 64, 16, "f16"),
        # a serving step's new tokens of a large mixed batch
        _case("append_step", "append", 256, 1, 1, 28, 4, 128, 32, "f16", rope=10000.0),
        # prompts of several requests prefilled together, odd lengths, with q/k norms
        _case("append_prompts", "append", 8, 509, 4096, 32, 8, 128, 16, "bf16", rope=500000.0,
              norm=True),
        # the smallest decode: two short sequences
        _case("decode_tiny", "decode", 2, 37, 100, 4, 2, 64, 16, "f16"),
        # an ordinary decode batch
        _case("decode_llama3_8b", "decode", 32, 512, 4096, 32, 8, 128, 16, "bf16"),
        # long contexts, few sequences
        _case("decode_long", "decode", 8, 32768, 32768, 32, 8, 128, 16, "bf16"),
        # a large batch of very uneven lengths, padded slots among it
        _case("decode_mixed", "decode", 256, 16, 8192, 28, 4, 128, 32, "f16", empty=3),
        # verifying drafts: a few tokens a sequence
        _case("multi_draft", "multi", 32, 512, 4096, 32, 8, 128, 16, "bf16", queries=5),
        # the end of long prompts: 64 tokens a sequence over a cached prefix
        _case("multi_suffix", "multi", 4, 1000, 8192, 32, 8, 128, 16, "bf16", queries=64),
        # the smallest serving step
        _case("step_tiny", "step", 2, 37, 100, 4, 2, 64, 16, "f16"),
        # an ordinary serving step: norm, rotation, append, decode
        _case("step_llama3_8b", "step", 32, 512, 4096, 32, 8, 128, 16, "bf16", rope=500000.0,
              norm=True),
        # a large uneven batch with padded slots
        _case("step_mixed", "step", 256, 16, 8192, 28, 4, 128, 32, "f16", rope=10000.0, empty=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "multi", "step"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16])
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "f16"])
    rope = rng.choice([0.0, 10000.0, 500000.0]) if op in ("append", "step") else 0.0
    norm = rope > 0.0 and rng.random() < 0.4
    batch = _log(rng, 1, 256)
    queries = 1
    if op == "append":
        # at most about the listed prompts' elements
        cap = max(1, 8 * 2000 * 48 * 128 // (batch * (group * hkv + 2 * hkv) * d))
        hi = _log(rng, 1, min(4096, cap))
        lo = _log(rng, 1, hi)
    else:
        # padded elements of one side: at most the listed long contexts'
        cap = 8 * 32768 * 8 * 128 // (batch * hkv * d)
        if op == "multi":
            queries = _log(rng, 2, 64)
            # scores of the plain form: at most the listed suffixes'
            cap = min(cap, 4 * 64 * 32 * 8192 // (batch * queries * group * hkv))
        hi = _log(rng, min(queries + 1, max(1, cap)), max(1, min(32768, cap)))
        lo = _log(rng, max(1, hi // 64), hi)
    empty = rng.choice([0, 0, 1]) if batch > 2 and op in ("decode", "step") else 0
    return _case("", op, batch, lo, hi, group * hkv, hkv, d, page, dtype, queries, rope, norm,
                 empty)


def _lens(c):
    """The case's lengths (tokens attended, or new tokens of an append): spread
    evenly over the logarithm from lo to hi; `empty` sequences have none."""
    n = c["batch"]
    r = c["hi"] / c["lo"]
    lens = [int(round(c["lo"] * r ** (i / max(1, n - 1)))) for i in range(n)]
    lens[-1] = c["hi"]
    for i in range(c["empty"]):
        lens[i] = 0
    return lens


def work(case):
    c = case
    lens = _lens(c)
    row = c["d"] * c["hkv"]          # elements of one token's K (or V)
    qrow = c["d"] * c["hq"]
    blocks = sum(-(-n // BLOCK) for n in lens)
    read8 = sum(lens) * row * 2 + blocks * c["hkv"] * 2
    per_query = 4 * c["d"] * c["hq"]  # two products a (query, key) pair
    if c["op"] == "append":
        t = sum(lens)
        rot = 2 * qrow * 2 if c["rope"] else 0
        return {"bytes": t * (2 * row * 2 + 2 * row + rot), "flops": t * (qrow + row) * 3}
    if c["op"] == "multi":
        m = c["queries"]
        pairs = sum(sum(max(0, n - m + j + 1) for j in range(m)) for n in lens)
        return {"bytes": read8 + 2 * 2 * qrow * m * len(lens), "flops": per_query * pairs}
    new = sum(1 for n in lens if n) * row * (4 + 2) if c["op"] == "step" else 0
    return {"bytes": read8 + 2 * 2 * qrow * len(lens) + new, "flops": per_query * sum(lens)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _need(a):
    """The smallest e with a <= 448 * 2^e, within the range of the scales."""
    f, e = torch.frexp(a)  # a = f 2^e, f in [0.5, 1); 448 = 0.875 * 2^9
    n = torch.where(f <= 0.875, e - 9, e - 8)
    return torch.where(a > 0, n.clamp(E_MIN, E_MAX), torch.full_like(n, E_MIN))


def _cache_side(x):
    """x [pages, heads, page, d] in fp32 -> (e4m3, exponents [pages, heads, blocks])."""
    n, h, p, d = x.shape
    b = x.reshape(n, h, p // BLOCK, BLOCK, d)
    e = _need(b.abs().amax((3, 4)))
    y = torch.ldexp(b, -e[..., None, None])
    return y.to(torch.float8_e4m3fn).reshape(n, h, p, d), e


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    B, P, D, Hq, Hkv = c["batch"], c["page"], c["d"], c["hq"], c["hkv"]
    lens = torch.tensor(_lens(c))[torch.randperm(B, generator=host)]
    if c["op"] == "append":  # new tokens after a cached start, which ends anywhere in a block
        start = torch.randint(0, 40, (B,), generator=host)
    else:
        start = torch.zeros(B, dtype=torch.int64)
    total = start + lens
    pages = (total + P - 1) // P
    most = (lens + (39 if c["op"] == "append" else 0) + P - 1) // P
    NP = int(most.sum()) + 2
    cols = max(1, int(most.max()))
    ids = torch.randperm(NP, generator=host).to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32)
    fill = torch.arange(cols)[None, :] < pages[:, None]
    table[fill] = ids[:int(pages.sum())]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    # the cache as earlier appends left it; heads differ in size, as they do in a model
    size = torch.exp2(torch.randint(-2, 3, (1, Hkv, 1, 1), generator=gen, device=dev).float())
    k_pool, ek = _cache_side(randn(NP, Hkv, P, D))
    v_pool, ev = _cache_side(randn(NP, Hkv, P, D) * size)
    scales = (torch.stack([ek, ev], -1) + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    s = dict(case=c, k_pool=k_pool, v_pool=v_pool, scales=scales, table=table.to(dev),
             scale=1.0 / math.sqrt(D), theta=c["rope"], eps=1e-6)
    if c["norm"]:
        s["q_norm"] = (1 + 0.1 * randn(D)).to(dt)
        s["k_norm"] = (1 + 0.1 * randn(D)).to(dt)
    else:
        s["q_norm"] = s["k_norm"] = None
    tokens = int(lens.sum()) if c["op"] == "append" else B
    if c["op"] == "append":
        seq = torch.repeat_interleave(torch.arange(B), lens)
        first = torch.cumsum(lens, 0) - lens
        pos = start[seq] + torch.arange(tokens) - first[seq]
        s["seq"] = seq.to(torch.int32).to(dev)
        # one new token of every sequence: the call needs no list of sequences
        s["single"] = bool((lens == 1).all())
    else:
        pos = lens - 1  # -1: a padded slot
        s["lens"] = lens.to(torch.int32).to(dev)
    s["pos"] = pos.to(torch.int32).to(dev)
    if c["op"] in ("append", "step"):
        s["k_new"] = randn(tokens, Hkv, D).to(dt)
        s["v_new"] = (randn(tokens, Hkv, D) * size.view(1, Hkv, 1)).to(dt)
    shape = (B, c["queries"], Hq, D) if c["op"] == "multi" else (tokens, Hq, D)
    s["q"] = randn(*shape).to(dt)
    s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _angles(s, d):
    inv = s["theta"] ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    a = s["pos"].double()[:, None] * inv
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _norm_rope(x, weight, s):
    """x [tokens, heads, d] in fp32: RMS norm of each head (where there is a
    weight), then the rotation of element i with element i + d/2."""
    if weight is not None:
        x = x * (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * weight.float()
    if s["theta"]:
        c, n = _angles(s, x.shape[-1])
        a, b = x.chunk(2, -1)
        x = torch.cat([a * c - b * n, b * c + a * n], -1)
    return x


def _append_side(x, pool, e_old, rows, blocks, fresh, slots):
    """x [tokens, heads, d] in fp32 into pool [pages, heads, page, d] (in place);
    e_old [blocks, heads] exponents; returns the new ones.  rows / blocks: each
    token's row ([page * slot]) and block; fresh [blocks]: the run starts at the
    block's first slot; slots [blocks]: slots in use before the run."""
    n_p, h, p, d = pool.shape
    a = torch.zeros(e_old.shape, device=x.device).scatter_reduce(
        0, blocks[:, None].expand(-1, h), x.abs().amax(-1), "amax")
    need = _need(a)
    touched = torch.zeros(e_old.shape[0], dtype=torch.bool, device=x.device)
    touched[blocks] = True
    e = torch.where(fresh[:, None], need, torch.maximum(e_old, need))
    e = torch.where(touched[:, None], e, e_old)
    ids = torch.unique(blocks)
    # earlier rows of the touched blocks, to the new scale
    page, blk = ids // (p // BLOCK), ids % (p // BLOCK)
    at = (blk[:, None] * BLOCK + torch.arange(BLOCK, device=x.device))[:, None, :]
    heads = torch.arange(h, device=x.device)[None, :, None]
    bits = pool.view(torch.uint8)
    old = bits[page[:, None, None], heads, at]
    y = torch.ldexp(old.view(torch.float8_e4m3fn).float(),
                    (e_old - e)[ids][..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    live = torch.arange(BLOCK, device=x.device)[None, :] < slots[ids][:, None]
    live &= ~fresh[ids][:, None]
    bits[page[:, None, None], heads, at] = torch.where(live[:, None, :, None], y, old)
    new = torch.ldexp(x, -e[blocks][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    bits[rows // p, :, rows % p] = new
    return e


def _plain_append(s, k, v):
    c = s["case"]
    P = c["page"]
    seq = s["seq"].long() if "seq" in s else torch.arange(c["batch"], device="cuda")
    pos = s["pos"].long()
    use = pos >= 0
    seq, pos, k, v = seq[use], pos[use], k[use], v[use]
    page = s["table"][seq, pos // P].long()
    rows = page * P + pos % P
    blocks = rows // BLOCK
    n = s["scales"].shape[0] * (P // BLOCK)
    # slots in use before the run: its first token's slot
    slots = torch.full((n,), BLOCK, device="cuda").scatter_reduce(0, blocks, pos % BLOCK, "amin")
    fresh = slots == 0
    e = s["scales"].view(torch.uint8).int() - 127  # [pages, heads, blocks of a page, side]
    e = e.permute(0, 2, 1, 3).reshape(n, c["hkv"], 2)
    ek = _append_side(k, s["k_pool"], e[..., 0], rows, blocks, fresh, slots)
    ev = _append_side(v, s["v_pool"], e[..., 1], rows, blocks, fresh, slots)
    e = torch.stack([ek, ev], -1).reshape(-1, P // BLOCK, c["hkv"], 2).permute(0, 2, 1, 3) + 127
    s["scales"].view(torch.uint8).copy_(e.to(torch.uint8))


def _dense(pool, e, table):
    """The cached values, [batch, heads, tokens, d] in fp32."""
    n, h, p, d = pool.shape
    t = table.clamp(min=0).long()
    x = pool.view(torch.uint8)[t].view(torch.float8_e4m3fn).float()
    x = x.reshape(*t.shape, h, p // BLOCK, BLOCK, d) * torch.exp2(e[t].float())[..., None, None]
    return x.permute(0, 2, 1, 3, 4, 5).reshape(t.shape[0], h, -1, d)


def _plain_attention(s, q):
    """q [batch, queries, heads, d] in fp32 -> the same shape."""
    c = s["case"]
    B, Q, Hq, D = q.shape
    H, G = c["hkv"], c["hq"] // c["hkv"]
    e = s["scales"].view(torch.uint8).int() - 127
    k = _dense(s["k_pool"], e[..., 0], s["table"])
    T = k.shape[2]
    qg = q.reshape(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    x = (qg @ k.transpose(2, 3)).reshape(B, H, G, Q, T) * s["scale"]
    del k
    last = s["lens"].long()[:, None] - Q + torch.arange(Q, device="cuda")
    see = torch.arange(T, device="cuda") <= last[..., None]
    x.masked_fill_(~see[:, None, None], float("-inf"))
    x -= x.amax(-1, keepdim=True).clamp(min=-1e30)
    x.exp_()
    den = x.sum(-1, keepdim=True)
    v = _dense(s["v_pool"], e[..., 1], s["table"])
    v.masked_fill_((torch.arange(T, device="cuda") >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = (x.reshape(B, H, G * Q, T) @ v).reshape(B, H, G, Q, D)
    o = torch.where(den > 0, o / den, torch.zeros_like(o))
    return o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)


def _plain(s):
    c = s["case"]
    dt = s["q"].dtype
    q = s["q"].float()
    if c["op"] in ("append", "step"):
        _plain_append(s, _norm_rope(s["k_new"].float(), s["k_norm"], s), s["v_new"].float())
        if s["theta"]:
            q = _norm_rope(q, s["q_norm"], s)
    cache = {"k_pool": s["k_pool"], "v_pool": s["v_pool"], "scales": s["scales"]}
    if c["op"] == "append":
        return dict(cache, q=q.to(dt)) if s["theta"] else cache
    if c["op"] == "multi":
        return {"out": _plain_attention(s, q).to(dt)}
    out = _plain_attention(s, q[:, None])[:, 0].to(dt)
    return {"out": out} if c["op"] == "decode" else dict(cache, out=out)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import paged_kv_decode_16_gb300 as pkv
    c = s["case"]
    cache = {"k_pool": s["k_pool"], "v_pool": s["v_pool"], "scales": s["scales"]}
    if c["op"] == "append":
        pool = s.get("pool")
        if pool is None:
            n, h, p, d = s["k_pool"].shape
            pool = s["pool"] = pkv.kv8_pool_create(n, p, h, d, s["k_pool"], s["v_pool"],
                                                   s["scales"])
        seq = None if s["single"] else s["seq"]
        if not s["theta"]:
            pkv.kv8_append(pool, s["k_new"], s["v_new"], s["table"], s["pos"], seq)
            return cache
        pkv.kv8_append_rope(pool, s["q"], s["k_new"], s["v_new"], s["table"], s["pos"],
                            s["theta"], s["out"], seq, q_norm_weight=s["q_norm"],
                            k_norm_weight=s["k_norm"], norm_eps=s["eps"])
        return dict(cache, q=s["out"])
    ws = s.get("workspace")
    if ws is None:
        ws = s["workspace"] = pkv.alloc_kv8_workspace(c["batch"], c["hq"], c["hkv"], c["d"],
                                                      n_queries=c["queries"])
    if c["op"] == "step":
        pkv.paged_decode_step_kv8(s["k_new"], s["v_new"], s["pos"], s["q"], s["k_pool"],
                                  s["v_pool"], s["scales"], s["table"], s["lens"], s["scale"],
                                  s["out"], ws, rope_theta=s["theta"], q_norm_weight=s["q_norm"],
                                  k_norm_weight=s["k_norm"], norm_eps=s["eps"])
        return dict(cache, out=s["out"])
    call = (pkv.paged_decode_attention_multi_kv8 if c["op"] == "multi"
            else pkv.paged_decode_attention_kv8)
    call(s["q"], s["k_pool"], s["v_pool"], s["scales"], s["table"], s["lens"], s["scale"],
         s["out"], ws)
    return {"out": s["out"]}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits, a sequence at a time
# ---------------------------------------------------------------------------
def _e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even), |x| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_rows(x, weight, theta, eps, pos):
    x = x.double()
    d = x.shape[-1]
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + eps) * weight.double()
    if theta:
        i = torch.arange(d // 2, device=x.device, dtype=torch.float64)
        ang = pos.double().view(-1, 1, 1) * torch.exp(i * (-2.0 / d * math.log(theta)))
        z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * torch.polar(torch.ones_like(ang), ang)
        x = torch.cat([z.real, z.imag], -1)
    return x


def _exact_append(s, k, v, kp, vp, e):
    """Run by run: kp, vp [pages, heads, page, d] and e [pages, heads, blocks, 2],
    in 64 bits, in place."""
    c = s["case"]
    P = c["page"]
    pos = s["pos"].tolist()
    seq = s["seq"].tolist() if "seq" in s else list(range(c["batch"]))
    table = s["table"].tolist()
    i = 0
    while i < len(pos):
        if pos[i] < 0:
            i += 1
            continue
        j = i + 1
        while j < len(pos) and seq[j] == seq[i] and pos[j] % BLOCK:
            j += 1
        page, lo = table[seq[i]][pos[i] // P], pos[i] % P
        blk, first = lo // BLOCK, lo // BLOCK * BLOCK
        for side, (x, pool) in enumerate(((k, kp), (v, vp))):
            y = x[i:j].transpose(0, 1)  # [heads, run, d]
            a = y.abs().amax((1, 2))
            ratio, need = torch.frexp(a.clamp(min=2.0 ** -90) / 448)  # ratio 2^need
            need = torch.where(ratio == 0.5, need - 1, need).clamp(E_MIN, E_MAX).double()
            e_new = need if lo == first else torch.maximum(need, e[page, :, blk, side])
            up = torch.exp2(e[page, :, blk, side] - e_new).view(-1, 1, 1)
            pool[page, :, first:lo] = _e4m3(pool[page, :, first:lo] * up)
            pool[page, :, lo:lo + j - i] = _e4m3(y / torch.exp2(e_new).view(-1, 1, 1))
            e[page, :, blk, side] = e_new
        i = j


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    P, D, H = c["page"], c["d"], c["hkv"]
    G = c["hq"] // H
    q = s["q"].double()
    e = s["scales"].view(torch.uint8).double() - 127
    if c["op"] in ("append", "step"):
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        _exact_append(s, _exact_rows(s["k_new"], s["k_norm"], s["theta"], s["eps"], s["pos"]),
                      s["v_new"].double(), kp, vp, e)
        if s["theta"]:
            q = _exact_rows(s["q"], s["q_norm"], s["theta"], s["eps"], s["pos"])
        cache = {"k_pool": kp, "v_pool": vp, "scales": torch.exp2(e)}
        if c["op"] == "append":
            return dict(cache, q=q) if s["theta"] else cache
    else:
        kp, vp = s["k_pool"], s["v_pool"]
    if c["op"] != "multi":
        q = q[:, None]
    out = torch.zeros_like(q)
    Q = q.shape[1]
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :(n + P - 1) // P].long()

        def side(pool, k):
            x = pool.view(torch.uint8)[pages].view(pool.dtype) if pool.dtype != torch.float64 \
                else pool[pages]
            x = x.double() * torch.exp2(e[pages][..., k]).repeat_interleave(BLOCK, 2)[..., None]
            return x.transpose(0, 1).reshape(H, -1, D)[:, :n]

        kk, vv = side(kp, 0), side(vp, 1)
        for h in range(H):
            for g in range(h * G, h * G + G):
                x = q[b, :, g] @ kk[h].T * s["scale"]
                t = torch.arange(n, device="cuda")
                j = torch.arange(Q, device="cuda")[:, None]
                x = torch.where(t <= n - Q + j, x, -math.inf)
                p = torch.nan_to_num(torch.softmax(x, -1))  # a query before the first token: 0
                out[b, :, g] = p @ vv[h]
    if c["op"] == "multi":
        return {"out": out}
    out = out[:, 0]
    return {"out": out} if c["op"] == "decode" else dict(cache, out=out)

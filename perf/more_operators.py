"""Paged serving with selected pages: what is measured.

Operators, in the order in which a step uses them:

  tables  page tables, slots and positions of a batch's new tokens, on the GPU,
          from the requests' lengths and a list of free pages
  append  rotary embedding (half or interleaved pairs, part of the head, scaled
          for long contexts, after an optional norm) of new tokens' q and k, and
          the write of k and v into their slots of the cache
  bounds  the smallest and the largest key of every page that got new tokens,
          channel by channel
  select  the pages that a query token attends to: the first and the last ones,
          and of the others those with the highest bound on q . k
  attend  decode attention over the selected pages
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, batch, lo, hi, hq=32, hkv=8, d=128, page=16, dtype="bf16", **more):
    c = dict(op=op, batch=batch, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, **more)
    return dict(c, name=name) if name else c


def _rope(rdim, inter=False, scaling="none", theta=500000.0, factor=1.0, low=1.0, high=4.0,
          context=8192, magnitude=1.0):
    return dict(rdim=rdim, inter=inter, scaling=scaling, theta=theta, factor=factor, low=low,
                high=high, context=context, magnitude=magnitude)


def listed():
    return [
        # the tables of a decode step: one new token for each running request
        _case("tables_step", "tables", 64, 1, 1, cached=4096, pad=0),
        # requests that decode and new prompts beside them, in one batch of a fixed size
        _case("tables_prompts", "tables", 256, 1, 8192, cached=8192, pad=777),
        # one token of one request: the smallest append
        _case("append_token", "append", 1, 1, 1, 4, 2, 64, 16, "f16", cached=100, pad=0,
              norm=False, fused=False, **_rope(64, theta=10000.0)),
        # a step of a large batch: interleaved pairs on half of the head, positions
        # stretched, rows of one fused projection, padded tokens behind the last
        _case("append_step", "append", 256, 1, 1, 28, 4, 128, 32, "f16", cached=30000, pad=7,
              norm=False, fused=True, **_rope(64, True, "linear", 10000.0, 4.0)),
        # prompts of several requests, odd lengths: norms, frequencies scaled by parts
        _case("append_prompts", "append", 8, 509, 4096, cached=3000, pad=0, norm=True, fused=True,
              **_rope(128, False, "turns", factor=8.0)),
        # the bounds of a decode step's pages
        _case("bounds_step", "bounds", 32, 1, 1, cached=4096, pad=0),
        # the bounds of whole prompts
        _case("bounds_prompts", "bounds", 32, 509, 8192, cached=100, pad=3),
        # the smallest selection: two short requests
        _case("select_tiny", "select", 2, 300, 1000, 4, 2, 64, 16, "f16", keep=8, empty=0),
        # an ordinary batch of long requests
        _case("select_long", "select", 32, 4096, 32768, keep=64, empty=1),
        # the smallest attention over selected pages
        _case("attend_tiny", "attend", 2, 300, 1000, 4, 2, 64, 16, "f16", keep=8, empty=0),
        # an ordinary batch: 64 pages of each request's 256 to 2048
        _case("attend_long", "attend", 32, 4096, 32768, keep=64, empty=1),
        # a large batch of uneven requests, larger pages, odd groups
        _case("attend_mixed", "attend", 256, 100, 16384, 28, 4, 128, 32, "f16", keep=40, empty=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "bounds", "select", "select", "attend",
                     "attend"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16])
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "f16"])
    batch = _log(rng, 1, 256)
    shape = (group * hkv, hkv, d, page, dtype)
    if op in ("tables", "append", "bounds"):
        # new tokens: at most about those of the listed prompts
        row = {"tables": 1, "append": (group + 2) * hkv * d, "bounds": hkv * d * 2}[op]
        most = {"tables": 50000, "append": 13000 * 48 * 128, "bounds": 80000 * 8 * 128 * 2}[op]
        hi = _log(rng, 1, max(1, min(8192, most // (row * batch))))
        lo = _log(rng, 1, hi)
        cached = _log(rng, 16, 30000 if op == "append" else 8192)
        if op == "bounds":  # the pool holds the cached tokens too
            cached = min(cached, max(1, most // (row * batch)))
        pad = rng.choice([0, 0, rng.randrange(1, 100)])
        more = {}
        if op == "append":
            rdim = rng.choice([16, 32, 64, d, d])
            scaling = rng.choice(["none", "none", "linear", "turns", "index"])
            more = dict(norm=rng.random() < 0.3, fused=rng.random() < 0.5,
                        **_rope(rdim, rng.random() < 0.4, scaling,
                                rng.choice([10000.0, 500000.0]),
                                1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                                high=32.0 if scaling == "index" else 4.0,
                                context=rng.choice([4096, 8192]),
                                magnitude=1.25 if scaling == "index" else 1.0))
        return _case("", op, batch, lo, hi, *shape, cached=cached, pad=pad, **more)
    empty = rng.choice([0, 0, 1]) if batch > 2 else 0
    if op == "select":
        cap = 32 * 32768 * 8 * 128 // 16 // (batch * hkv * d) * page // 3
        hi = _log(rng, 16 * page, max(16 * page, min(131072, cap)))
        keep = _log(rng, 4, max(4, min(128, hi // page // 2)))
    else:
        # elements of one side that are read: at most those of the listed uneven batch
        most = 200 * 1024 * 4 * 128 // max(1, group // 8)
        keep = max(2, min(_log(rng, 4, 128), most // (batch * hkv * d * page)))
        hi = _log(rng, 1, max(16, min(65536, 32 * 32768 * 8 * 128 // (batch * hkv * d))))
    lo = _log(rng, max(1, hi // 64), hi)
    return _case("", op, batch, lo, hi, *shape, keep=keep, empty=empty)


def _lens(c):
    """The case's lengths (tokens attended, or new tokens): spread evenly over the
    logarithm from lo to hi; `empty` requests have none."""
    n = c["batch"]
    r = c["hi"] / c["lo"]
    lens = [int(round(c["lo"] * r ** (i / max(1, n - 1)))) for i in range(n)]
    lens[-1] = c["hi"]
    if c["op"] == "tables" and c["hi"] > 1:  # seven of eight only decode
        lens = [m if i % 8 == 7 else 1 for i, m in enumerate(lens)]
    for i in range(c.get("empty", 0)):
        lens[i] = 0
    return lens


def _kept(c):
    """Pages always listed: the first ones and the last ones."""
    return (1, 2) if c["keep"] >= 4 else (0, 1)


def work(case):
    c = case
    lens = _lens(c)
    P, D, Hq, Hkv, B = c["page"], c["d"], c["hq"], c["hkv"], c["batch"]
    t = sum(lens)
    if c["op"] == "tables":
        return {"bytes": 8 * B + 4 * B + 4 * (B + 1) + 16 * (t + c["pad"]) + 8 * (t // P + B),
                "flops": 8 * t}
    if c["op"] == "append":
        return {"bytes": t * ((Hq + 2 * Hkv) * D * 4 + 12), "flops": t * (Hq + Hkv) * c["rdim"] * 3}
    if c["op"] == "bounds":
        # the pages' rows: the new ones and, at worst, a page's older ones
        pages = sum(-(-n // P) for n in lens)
        return {"bytes": t * Hkv * D * 2 + pages * Hkv * 2 * D * 2 + 8 * t,
                "flops": 2 * t * Hkv * D}
    pages = [-(-n // P) for n in lens]
    lists = 4 * B * Hkv * c["keep"]
    if c["op"] == "select":
        first, last = _kept(c)
        scored = sum(n - first - last for n in pages if n > c["keep"])
        return {"bytes": scored * Hkv * (2 * D * 2) + B * Hq * D * 2 + lists + 4 * sum(pages),
                "flops": scored * Hq * D * 4}
    read = sum(min(n, c["keep"] * P - (-n) % P) for n in lens)
    return {"bytes": read * Hkv * D * 4 + 2 * B * Hq * D * 2 + lists, "flops": read * Hq * D * 4}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    op, B, P, D, Hq, Hkv = c["op"], c["batch"], c["page"], c["d"], c["hq"], c["hkv"]
    lens = torch.tensor(_lens(c))[torch.randperm(B, generator=host)]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def i32(x):
        return x.to(torch.int32).to(dev)

    s = dict(case=c)
    if op in ("tables", "append", "bounds"):
        # new tokens behind what earlier steps cached
        cached = torch.randint(0, c["cached"] + 1, (B,), generator=host)
        old, total = -(-cached // P), -(-(cached + lens) // P)
        tokens = int(lens.sum())
        n_old = int(old.sum())
        # sizes go by the longest that a request may be; an append has only the pages that
        # get tokens, however far their positions are
        low = cached // P if op == "append" else torch.zeros_like(cached)
        most = lens + (P - 1 if op == "append" else c["cached"])
        NP = int((-(-most // P)).sum()) + 64
        ids = torch.randperm(NP, generator=host)
        cols = -(-(c["cached"] + c["hi"]) // P)
        if op == "tables":
            table = torch.full((B, cols), -1, dtype=torch.int32)
            table[torch.arange(cols)[None, :] < old[:, None]] = ids[:n_old].to(torch.int32)
            begin = 3  # pages that earlier calls took from the list
            free = torch.cat([ids[:begin], ids[n_old:]])
            s.update(cached=i32(cached), new=i32(lens), free=i32(free),
                     begin=i32(torch.tensor([begin])), end=i32(torch.zeros(1)), table=table.to(dev),
                     pages=NP, lens=i32(torch.zeros(B)), starts=i32(torch.zeros(B + 1)),
                     pos=i32(torch.zeros(tokens + c["pad"])), seq=i32(torch.zeros(tokens + c["pad"])),
                     slots=torch.zeros(tokens + c["pad"], dtype=torch.int64, device=dev))
            return s
        seq = torch.repeat_interleave(torch.arange(B), lens)
        first = torch.cumsum(lens, 0) - lens
        pos = cached[seq] + torch.arange(tokens) - first[seq]
        base = torch.cumsum(total - low, 0) - (total - low)
        page = ids[base[seq] + pos // P - low[seq]]
        none = torch.full((c["pad"],), -1, dtype=torch.int64)
        s["pos"] = i32(torch.cat([pos, none]))
        s["slots"] = torch.cat([page * P + pos % P, none]).to(dev)
        n = tokens + c["pad"]
        if op == "bounds":
            s["k_pool"] = randn(NP, Hkv, P, D).to(dt)
            s["v_pool"] = s["k_pool"]  # not read
            s["bounds"] = torch.zeros(NP, Hkv, 2, D, dtype=dt, device=dev)
            return s
        s["k_pool"] = torch.zeros(NP, Hkv, P, D, dtype=dt, device=dev)
        s["v_pool"] = torch.zeros(NP, Hkv, P, D, dtype=dt, device=dev)
        if c["fused"]:  # the rows of one projection of the hidden state
            x = randn(n, Hq + 2 * Hkv, D).to(dt)
            s["q"], s["k"], s["v"] = x.split([Hq, Hkv, Hkv], 1)
        else:
            s["q"], s["k"], s["v"] = (randn(n, h, D).to(dt) for h in (Hq, Hkv, Hkv))
        s["out"] = torch.zeros(n, Hq, D, dtype=dt, device=dev)
        s["eps"] = 1e-6
        s["q_norm"] = s["k_norm"] = None
        if c["norm"]:
            s["q_norm"] = (1 + 0.1 * randn(D)).to(dt)
            s["k_norm"] = (1 + 0.1 * randn(D)).to(dt)
        return s

    pages = -(-lens // P)
    NP, cols = int(pages.sum()) + 2, max(1, int(pages.max()))
    table = torch.full((B, cols), -1, dtype=torch.int32)
    fill = torch.arange(cols)[None, :] < pages[:, None]
    table[fill] = torch.randperm(NP, generator=host)[:NP - 2].to(torch.int32)
    s.update(table=table.to(dev), lens=i32(lens), q=randn(B, Hq, D).to(dt), scale=D ** -0.5)
    K = c["keep"]
    s["sel"] = torch.full((B, Hkv, K), -1, dtype=torch.int32, device=dev)
    if op == "select":
        # the keys of a page lie together: around a centre of its own
        mid = 0.7 * randn(NP, Hkv, 1, D)
        half = torch.rand(NP, Hkv, 1, D, generator=gen, device=dev) + 0.8
        s["bounds"] = torch.cat([mid - half, mid + half], 2).to(dt)
        return s
    # lists as a selection makes them: the first page, the last two, others at random
    first, last = _kept(c)
    n = pages.to(dev)[:, None, None]
    j = torch.arange(cols, device=dev)
    score = torch.rand(B, Hkv, cols, generator=gen, device=dev)
    score = torch.where((j < first) | (j >= n - last), 2.0, score)
    score = torch.where(j < n, score, -1.0)
    k = min(K, cols)
    val, at = score.topk(k, -1)
    at = torch.where(val < 0, cols, at).sort(-1).values
    s["sel"][..., :k] = torch.where(at < cols, at, -1).to(torch.int32)
    s["k_pool"] = randn(NP, Hkv, P, D).to(dt)
    s["v_pool"] = randn(NP, Hkv, P, D).to(dt)
    s["out"] = torch.empty(B, Hq, D, dtype=dt, device=dev)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _frequencies(c):
    """Radians a position for each rotated pair."""
    r, base = c["rdim"], c["theta"]
    inv = [base ** (-2.0 * i / r) for i in range(r // 2)]
    f = c["factor"]
    if c["scaling"] == "linear":
        return [x / f for x in inv]
    if c["scaling"] == "turns":  # pairs of few turns over the original context are stretched
        out = []
        for x in inv:
            n = c["context"] * x / (2 * math.pi)
            g = min(1.0, max(0.0, (n - c["low"]) / (c["high"] - c["low"])))
            out.append((1 - g) * x / f + g * x)
        return out
    if c["scaling"] == "index":  # the same with a ramp over the pairs' indexes
        def at(n):
            return r * math.log(c["context"] / (2 * math.pi * n)) / (2 * math.log(base))
        lo = max(math.floor(at(c["high"])), 0)
        hi = min(math.ceil(at(c["low"])), r - 1)
        hi = max(hi, lo + 0.001)
        ramp = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(r // 2)]
        return [x / f * g + x * (1 - g) for x, g in zip(inv, ramp)]
    return inv


def _plain_tables(s):
    c = s["case"]
    P = c["page"]
    cached, new = s["cached"].long(), s["new"].long()
    old, total = (cached + P - 1) // P, (cached + new + P - 1) // P
    need = total - old
    upto = torch.cumsum(need, 0)
    begin = s["begin"].long()
    j = torch.arange(s["table"].shape[1], device="cuda")
    take = (begin + (upto - need))[:, None] + j - old[:, None]
    fresh = s["free"][take.clamp(0, s["free"].shape[0] - 1)]
    mine = (j >= old[:, None]) & (j < total[:, None])
    s["table"].copy_(torch.where(mine, fresh, s["table"]))
    s["end"].copy_(begin + upto[-1:])
    s["lens"].copy_(cached + new)
    ends = torch.cumsum(new, 0)
    s["starts"][0] = 0
    s["starts"][1:] = ends
    i = torch.arange(s["pos"].shape[0], device="cuda")
    seq = torch.searchsorted(ends, i, right=True).clamp(max=c["batch"] - 1)
    pos = cached[seq] + i - (ends - new)[seq]
    live = i < ends[-1]
    page = s["table"][seq, torch.where(live, pos // P, 0)].long()
    s["pos"].copy_(torch.where(live, pos, -1))
    s["seq"].copy_(torch.where(live, seq, -1))
    s["slots"].copy_(torch.where(live, page * P + pos % P, -1))


def _plain_rotate(x, weight, s):
    """x [tokens, heads, d] in fp32."""
    c = s["case"]
    r = c["rdim"]
    if weight is not None:
        x = x * (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * weight.float()
    inv = torch.tensor(_frequencies(c), dtype=torch.float64, device="cuda")
    a = s["pos"].double()[:, None, None] * inv
    cos, sin = (a.cos() * c["magnitude"]).float(), (a.sin() * c["magnitude"]).float()
    y = x.clone()
    one, two = ((slice(0, r, 2), slice(1, r, 2)) if c["inter"]
                else (slice(0, r // 2), slice(r // 2, r)))
    y[..., one] = x[..., one] * cos - x[..., two] * sin
    y[..., two] = x[..., two] * cos + x[..., one] * sin
    return y


def _plain_append(s):
    P = s["case"]["page"]
    dt = s["q"].dtype
    live = s["pos"] >= 0
    q = _plain_rotate(s["q"].float(), s["q_norm"], s).to(dt)
    k = _plain_rotate(s["k"].float(), s["k_norm"], s).to(dt)
    s["out"].copy_(torch.where(live[:, None, None], q, s["out"]))
    at = s["slots"]
    use = at >= 0
    at, k, v = at[use], k[use], s["v"][use]
    s["k_pool"][at // P, :, at % P] = k
    s["v_pool"][at // P, :, at % P] = v


def _plain_bounds(s):
    P = s["case"]["page"]
    at = s["slots"][s["slots"] >= 0]
    rows = torch.zeros(s["bounds"].shape[0], dtype=torch.int64, device="cuda")
    rows.scatter_reduce_(0, at // P, at % P + 1, "amax")
    ids = torch.nonzero(rows)[:, 0]
    x = s["k_pool"][ids].float()
    out = (torch.arange(P, device="cuda") >= rows[ids, None])[:, None, :, None]
    lo = x.masked_fill(out, float("inf")).amin(2)
    hi = x.masked_fill_(out, float("-inf")).amax(2)
    s["bounds"][ids] = torch.stack([lo, hi], 2).to(s["bounds"].dtype)


def _plain_select(s):
    c = s["case"]
    B, Hkv, K = s["sel"].shape
    P, D = c["page"], c["d"]
    first, last = _kept(c)
    n = ((s["lens"].long() + P - 1) // P)[:, None, None]
    # 64 bits: the last page that is taken and the first that is not may be close
    q = s["q"].double().reshape(B, Hkv, -1, D)
    up, down = q.clamp(min=0), q.clamp(max=0)
    score = torch.empty(B, Hkv, s["table"].shape[1], dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        b = s["bounds"][s["table"].clamp(min=0).long(), h].double()  # [B, pages, 2, D]
        x = up[:, h] @ b[:, :, 1].transpose(1, 2) + down[:, h] @ b[:, :, 0].transpose(1, 2)
        score[:, h] = x.amax(1)
    j = torch.arange(score.shape[2], device="cuda")
    inf = float("inf")
    score = torch.where((j < first) | (j >= n - last), inf, score)
    score = torch.where(j < n, score, -inf)
    k = min(K, score.shape[2])
    at = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    at = torch.where(at < n, at, score.shape[2]).sort(-1).values
    s["sel"].fill_(-1)
    s["sel"][..., :k] = torch.where(at < n, at, -1)


def _plain_attend(s):
    c = s["case"]
    B, Hkv, K = s["sel"].shape
    P, D = c["page"], c["d"]
    dt = s["q"].dtype
    sel = s["sel"].long()
    page = s["table"].long()[torch.arange(B, device="cuda")[:, None, None], sel.clamp(min=0)]
    page = page.clamp(min=0)
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    tok = sel[..., None] * P + torch.arange(P, device="cuda")
    see = ((sel[..., None] >= 0) & (tok < s["lens"].long()[:, None, None, None]))
    see = see.reshape(B, Hkv, 1, K * P)
    q = s["q"].float().reshape(B, Hkv, -1, D)
    k = s["k_pool"][page, h].float().reshape(B, Hkv, K * P, D)
    x = (q @ k.transpose(2, 3)) * s["scale"]
    del k
    x.masked_fill_(~see, float("-inf"))
    x -= x.amax(-1, keepdim=True).clamp(min=-1e30)
    x.exp_()
    den = x.sum(-1, keepdim=True)
    v = s["v_pool"][page, h].float().reshape(B, Hkv, K * P, D)
    v.masked_fill_(~see.transpose(2, 3), 0.0)
    o = x @ v
    o = torch.where(den > 0, o / den, torch.zeros_like(o))
    s["out"].copy_(o.reshape(B, -1, D).to(dt))


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import paged_kv_decode_16_gb300 as pkv
    c = s["case"]
    op = c["op"]
    if op == "tables":
        pkv.paged_tables_build(s["cached"], s["new"], s["free"], s["begin"], s["end"], s["table"],
                               c["page"], s["pages"], s["lens"], s["starts"], s["pos"], s["seq"],
                               s["slots"])
    elif op == "append" or op == "bounds":
        pool = s.get("pool")
        if pool is None:
            n, h, p, d = s["k_pool"].shape
            pool = s["pool"] = pkv.kv_pool_create(n, p, h, d, s["k_pool"].dtype, s["k_pool"],
                                                  s["v_pool"])
        if op == "bounds":
            pkv.kv_page_bounds(pool, s["slots"], s["bounds"])
            return
        rope = s.get("rope")
        if rope is None:
            rope = s["rope"] = pkv.Rope(c["rdim"], c["theta"], interleaved=c["inter"],
                                        scaling=c["scaling"], factor=c["factor"],
                                        low_turns=c["low"], high_turns=c["high"],
                                        original_context=c["context"], magnitude=c["magnitude"])
        pkv.kv_append_tokens(pool, s["k"], s["v"], s["slots"], q=s["q"], positions=s["pos"],
                             rope=rope, q_out=s["out"], q_norm_weight=s["q_norm"],
                             k_norm_weight=s["k_norm"], norm_eps=s["eps"])
    elif op == "select":
        first, last = _kept(c)
        ws = s.get("workspace")
        if ws is None:
            ws = s["workspace"] = pkv.alloc_select_workspace(c["batch"], c["hkv"],
                                                             s["table"].shape[1])
        pkv.paged_select_pages(s["q"], s["bounds"], s["table"], s["lens"], c["page"], s["sel"],
                               ws, keep_first=first, keep_last=last)
    else:
        pkv.paged_decode_attention_selected(s["q"], s["k_pool"], s["v_pool"], s["table"],
                                            s["lens"], s["sel"], s["scale"], s["out"])


def _results(s):
    op = s["case"]["op"]
    names = {"tables": ("table", "end", "lens", "starts", "pos", "seq", "slots"),
             "append": ("k_pool", "v_pool", "out"), "bounds": ("bounds",), "select": ("sel",),
             "attend": ("out",)}[op]
    return {k: s[k] for k in names}


def run(state):
    if own:
        _own(state)
    else:
        {"tables": _plain_tables, "append": _plain_append, "bounds": _plain_bounds,
         "select": _plain_select, "attend": _plain_attend}[state["case"]["op"]](state)
    return _results(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a request at a time
# ---------------------------------------------------------------------------
def _exact_tables(s):
    P = s["case"]["page"]
    cached, new, free = s["cached"].tolist(), s["new"].tolist(), s["free"].tolist()
    at = s["begin"].item()
    table = s["table"].tolist()
    lens, starts, pos, seq, slots = [], [0], [], [], []
    for b, (c, n) in enumerate(zip(cached, new)):
        for t in range(c, c + n):
            if t % P == 0:
                table[b][t // P] = free[at]
                at += 1
            pos.append(t)
            seq.append(b)
            slots.append(table[b][t // P] * P + t % P)
        lens.append(c + n)
        starts.append(starts[-1] + n)
    none = [-1] * s["case"]["pad"]
    res = dict(table=table, end=[at], lens=lens, starts=starts, pos=pos + none, seq=seq + none,
               slots=slots + none)
    return {k: torch.tensor(v, dtype=s[k].dtype, device="cuda") for k, v in res.items()}


def _exact_rows(x, weight, s):
    c = s["case"]
    x = x.double()
    r = c["rdim"]
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * weight.double()
    ang = s["pos"].double().view(-1, 1, 1) * torch.tensor(_frequencies(c), dtype=torch.float64,
                                                          device="cuda")
    turn = torch.polar(torch.full_like(ang, c["magnitude"]), ang)
    z, rest = x[..., :r], x[..., r:]
    if c["inter"]:
        z = torch.view_as_real(torch.view_as_complex(z.reshape(*z.shape[:-1], -1, 2).contiguous())
                               * turn).flatten(-2)
    else:
        z = torch.complex(z[..., :r // 2], z[..., r // 2:]) * turn
        z = torch.cat([z.real, z.imag], -1)
    return torch.cat([z, rest], -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op, P, D, H = c["op"], c["page"], c["d"], c["hkv"]
    G = c["hq"] // H
    if op == "tables":
        return _exact_tables(s)
    if op == "append":
        q, k = _exact_rows(s["q"], s["q_norm"], s), _exact_rows(s["k"], s["k_norm"], s)
        res = {n: s[n].double() for n in ("k_pool", "v_pool", "out")}
        n = c["pad"]
        m = q.shape[0] - n
        res["out"][:m] = q[:m]
        for pool, x in (("k_pool", k), ("v_pool", s["v"].double())):
            flat = res[pool].transpose(1, 2).reshape(-1, H, D)
            flat[s["slots"][:m]] = x[:m]
            res[pool] = flat.reshape(-1, P, H, D).transpose(1, 2)
        return res
    if op == "bounds":
        top = {}  # each page's rows in use
        for x in s["slots"].tolist():
            if x >= 0:
                top[x // P] = max(top.get(x // P, 0), x % P + 1)
        res = s["bounds"].double()
        for rows in set(top.values()):
            ids = torch.tensor([p for p, m in top.items() if m == rows], device="cuda")
            x = s["k_pool"][ids, :, :rows].double()
            res[ids, :, 0], res[ids, :, 1] = x.min(2).values, x.max(2).values
        return {"bounds": res}
    lens = s["lens"].tolist()
    if op == "select":
        first, last = _kept(c)
        res = torch.full_like(s["sel"], -1)
        K = c["keep"]
        for b, m in enumerate(lens):
            n = -(-m // P)
            if n <= K:
                res[b, :, :n] = torch.arange(n, device="cuda")
                continue
            bound = s["bounds"][s["table"][b, first:n - last].long()].double()
            for h in range(H):
                best = None
                for g in range(h * G, h * G + G):
                    q = s["q"][b, g].double()
                    x = torch.where(q >= 0, bound[:, h, 1], bound[:, h, 0]) @ q
                    best = x if best is None else torch.maximum(best, x)
                best = best.tolist()
                order = sorted(range(len(best)), key=lambda i: (-best[i], i))
                mid = sorted(i + first for i in order[:K - first - last])
                mid = list(range(first)) + mid + list(range(n - last, n))
                res[b, h] = torch.tensor(mid, dtype=torch.int32, device="cuda")
        return {"sel": res}
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    sel = s["sel"].tolist()
    for b, m in enumerate(lens):
        for h in range(H):
            ids = [j for j in sel[b][h] if j >= 0]
            if not ids or m == 0:
                continue
            at = s["table"][b, torch.tensor(ids, device="cuda")].long()
            n = sum(min(P, m - j * P) for j in ids)  # only the last page may be short
            k = s["k_pool"][at, h].double().reshape(-1, D)[:n]
            v = s["v_pool"][at, h].double().reshape(-1, D)[:n]
            q = s["q"][b, h * G:h * G + G].double()
            out[b, h * G:h * G + G] = torch.softmax(q @ k.T * s["scale"], -1) @ v
    return {"out": out}

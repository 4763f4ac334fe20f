"""Serving with selected pages on the GPU: every call against plain forms in 64 bits
(selected_ref.py), its refusals of data, streams and graphs, and a run of them together."""
import math
import random

import pytest
import torch

import paged_kv_decode_16_gb300 as pkv
import selected_ref as ref

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def i64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def rand(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device=DEV).to(dtype)


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------
def run_tables(cached, new, free, begin, table, page, num_pages, n_tokens, status=None,
               stream=None):
    B = len(cached)
    out = dict(table=i32(table).reshape(B, -1) if B else i32([]).reshape(0, 4),
               lens=i32([77] * B), starts=i32([77] * (B + 1)),
               pos=i32([77] * n_tokens), seq=i32([77] * n_tokens), slots=i64([77] * n_tokens),
               end=i32([77]))
    pkv.paged_tables_build(i32(cached), i32(new), i32(free), i32([begin]), out["end"],
                           out["table"], page, num_pages, out["lens"], out["starts"], out["pos"],
                           out["seq"], out["slots"], dev_status=status, stream=stream)
    return out


def check_tables(cached, new, free, begin, table, page, num_pages, n_tokens):
    st = status_word()
    got = run_tables(cached, new, free, begin, table, page, num_pages, n_tokens, st)
    want = ref.tables(cached, new, free, begin, table, page, num_pages, n_tokens)
    for name, w in zip(("table", "lens", "starts", "pos", "seq", "slots"), want):
        assert got[name].tolist() == w, name
    assert got["end"].tolist() == [want[6]]
    assert st.item() == want[7]
    return want[7]


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("page", [16, 48, 256])
def test_tables_of_random_batches(page, seed):
    rng = random.Random(100 * page + seed)
    B = [1, 3, 40, 257, 700, 33][seed]
    cols = rng.randrange(4, 20)
    cached = [rng.choice([0, 1, page - 1, page, rng.randrange(0, cols * page)]) for _ in range(B)]
    new = [min(rng.choice([0, 1, 1, page, rng.randrange(0, 3 * page)]), cols * page - c)
           for c in cached]
    need = [-(-(c + n) // page) - -(-c // page) for c, n in zip(cached, new)]
    total = sum(-(-c // page) for c in cached) + sum(need)
    ids = list(range(total + 10))
    rng.shuffle(ids)
    table, at = [], 0
    for c in cached:
        k = -(-c // page)
        table.append(ids[at:at + k] + [-5] * (cols - k))
        at += k
    free = [0, 0] + ids[at:]
    assert check_tables(cached, new, free, 2, table, page, total + 10,
                        sum(new) + rng.choice([0, 1, 2000])) == 0


@pytest.mark.parametrize("case,flag", [
    ("row", ref.BAD_LEN), ("tokens", ref.BAD_LEN), ("negative", ref.BAD_LEN),
    ("pages", ref.NO_PAGES), ("no pages at all", ref.NO_PAGES), ("begin", ref.NO_PAGES),
    ("old page", ref.BAD_PAGE), ("new page", ref.BAD_PAGE), ("huge", ref.BAD_LEN)])
def test_tables_refuse_requests(case, flag):
    cached, new = [5, 16, 31, 0, 20], [3, 1, 2, 20, 0]
    table = [[0, -1, -1], [1, -1, -1], [2, 3, -1], [-1, -1, -1], [4, 5, -1]]
    free, begin, tokens = [6, 7, 8, 9, 10], 1, 30
    if case == "row":
        new[2] = 18
    elif case == "tokens":
        tokens = 25
    elif case == "negative":
        cached[1], new[2] = -1, -3
    elif case == "pages":
        free = free[:3]
    elif case == "no pages at all":
        free, begin = [], 0
    elif case == "begin":
        begin = 6
    elif case == "old page":
        table[0][0] = 99
    elif case == "new page":
        free[1] = -2
    elif case == "huge":
        new[3] = 2 ** 31 - 1
        cached[4] = 2 ** 31 - 1
    assert check_tables(cached, new, free, begin, table, 16, 16, tokens) & flag


def test_tables_of_nothing():
    check_tables([], [], [1, 2], 1, [], 16, 8, 5)
    check_tables([3, 0], [0, 0], [], 0, [[1, 1], [1, 1]], 16, 8, 0)
    check_tables([0], [1], [3], 0, [[-1]], 16, 8, 1)


def test_tables_largest_batch():
    rng = random.Random(5)
    B = 16384
    cached = [rng.randrange(0, 40) for _ in range(B)]
    new = [rng.choice([0, 1, 1, 1, 5]) for _ in range(B)]
    ids = list(range(5 * B))
    rng.shuffle(ids)
    table = [[ids[3 * b], ids[3 * b + 1], ids[3 * b + 2]] for b in range(B)]
    assert check_tables(cached, new, ids[3 * B:], 0, table, 16, 5 * B, sum(new) + 3) == 0


def test_tables_of_millions_of_tokens():
    """Token sums of one round of the CTA beyond 32 bits' guard, many tokens a CTA."""
    new, page, cols = [4000001, 0, 1, 4900000], 256, 20000
    B, N = len(new), 9000000
    need = [-(-n // page) for n in new]
    order = torch.randperm(sum(need), device=DEV).to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    out = dict(lens=i32([0] * B), starts=i32([0] * (B + 1)), end=i32([0]),
               pos=torch.zeros(N, dtype=torch.int32, device=DEV),
               seq=torch.zeros(N, dtype=torch.int32, device=DEV),
               slots=torch.zeros(N, dtype=torch.int64, device=DEV))
    st = status_word()
    pkv.paged_tables_build(i32([0] * B), i32(new), order, None, out["end"], table, page,
                           sum(need), out["lens"], out["starts"], out["pos"], out["seq"],
                           out["slots"], dev_status=st)
    assert st.item() == 0 and out["end"].item() == sum(need) and out["lens"].tolist() == new
    assert out["starts"].tolist() == [0, 4000001, 4000001, 4000002, sum(new)]
    row = at = 0
    for b, n in enumerate(new):
        p = torch.arange(n, device=DEV)
        pages = order[at:at + need[b]].long()
        assert torch.equal(table[b, :need[b]].long(), pages) and (table[b, need[b]:] == -1).all()
        assert torch.equal(out["pos"][row:row + n].long(), p)
        assert (out["seq"][row:row + n] == b).all()
        assert torch.equal(out["slots"][row:row + n], pages[p // page] * page + p % page)
        row, at = row + n, at + need[b]
    for name in ("pos", "seq", "slots"):
        assert (out[name][row:] == -1).all()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def make_pool(num_pages, page, hkv, d, dtype, fill=7.0):
    k = torch.full((num_pages, hkv, page, d), fill, dtype=dtype, device=DEV)
    v = torch.full_like(k, -fill)
    return pkv.kv_pool_create(num_pages, page, hkv, d, dtype, k, v), k, v


def token_rows(gen, tokens, hq, hkv, d, dtype, fused):
    if fused:
        x = rand(gen, tokens, hq + 2 * hkv, d, dtype=dtype)
        return x.split([hq, hkv, hkv], 1)
    return tuple(rand(gen, tokens, h, d, dtype=dtype) for h in (hq, hkv, hkv))


def check_append(tokens, hq, hkv, d, page, dtype, rdim, inter, scaling, magnitude, norm, fused,
                 seed, in_place=False, most=200000):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    NP = tokens // page + 4
    pool, k_pool, v_pool = make_pool(NP, page, hkv, d, dtype)
    slots = rng.sample(range(NP * page), tokens)
    pos = [rng.choice([0, 1, most, rng.randrange(0, most)]) for _ in range(tokens)]
    for i in range(tokens):
        if rng.random() < 0.1:
            slots[i] = -1           # turned, not written
        if rng.random() < 0.1:
            pos[i] = -1             # skipped whole
    q, k, v = token_rows(gen, tokens, hq, hkv, d, dtype, fused)
    weights = [(1 + 0.2 * rand(gen, d, dtype=torch.float32)).to(dtype) if norm else None
               for _ in range(2)]
    kw = dict(theta=10000.0, interleaved=inter, scaling=scaling, factor=8.0, low_turns=1.0,
              high_turns=32.0, original_context=4096.0, magnitude=magnitude)
    freq = ref.frequencies(rdim, 10000.0, scaling, 8.0, 1.0, 32.0, 4096.0)
    p = torch.tensor(pos)
    want_q, err_q = ref.turned(q, p, freq, inter, magnitude, weights[0], 1e-6)
    want_k, err_k = ref.turned(k, p, freq, inter, magnitude, weights[1], 1e-6)
    q_out = q if in_place else torch.full((tokens, hq, d), 3.0, dtype=dtype, device=DEV)
    before, v0 = q_out.clone(), v.clone()
    st = status_word()
    res = pkv.kv_append_tokens(pool, k, v, i64(slots), q=q, positions=i32(pos),
                               rope=pkv.Rope(rdim, **kw), q_out=q_out, q_norm_weight=weights[0],
                               k_norm_weight=weights[1], norm_eps=1e-6, dev_status=st)
    assert res is q_out and st.item() == 0
    skip = p < 0
    assert torch.equal(q_out[skip.to(DEV)], before[skip.to(DEV)])
    ref.close(q_out[~skip.to(DEV)], want_q[~skip], ref.rounded(want_q, err_q, dtype)[~skip], "q")
    if not norm:  # what does not turn is copied
        assert torch.equal(q_out[~skip.to(DEV)][..., rdim:], (before if in_place else q)[
            ~skip.to(DEV)][..., rdim:])
    kp = torch.full((NP * page, hkv, d), 7.0, dtype=torch.float64)
    kb = torch.zeros_like(kp)
    vp = torch.full((NP * page, hkv, d), -7.0, dtype=dtype)
    for i, s in enumerate(slots):
        if s >= 0 and pos[i] >= 0:
            kp[s], kb[s] = want_k[i], ref.rounded(want_k[i], err_k[i], dtype)
            vp[s] = v0[i].cpu()
    flat = [x.transpose(1, 2).reshape(NP * page, hkv, d) for x in (k_pool, v_pool)]
    ref.close(flat[0], kp, kb, "k")
    assert torch.equal(flat[1].cpu(), vp)


@pytest.mark.parametrize("tokens", [1, 2, 7, 300, 2500])
@pytest.mark.parametrize("hq,hkv,d,page,dtype,rdim,inter,fused", [
    (4, 2, 64, 16, F16, 64, False, False),
    (32, 8, 128, 16, BF16, 128, False, True),
    (28, 4, 128, 32, F16, 64, True, True),
    (5, 5, 64, 48, BF16, 16, True, False),
    (12, 1, 128, 256, BF16, 112, False, True),
])
def test_append_turns_and_writes(tokens, hq, hkv, d, page, dtype, rdim, inter, fused):
    check_append(tokens, hq, hkv, d, page, dtype, rdim, inter, "none", 1.0, False, fused, tokens)


@pytest.mark.parametrize("scaling", ["linear", "turns", "index"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_append_scalings_and_norms(scaling, norm, inter):
    for dtype in (BF16, F16):
        check_append(37, 6, 3, 128, 16, dtype, 96, inter, scaling, 1.3, norm, True, 11)
        check_append(37, 6, 3, 64, 16, dtype, 64, inter, scaling, 0.7, norm, False, 12)


def test_append_far_positions():
    check_append(64, 4, 2, 128, 16, F16, 128, False, "none", 1.0, False, True, 3,
                 most=2 ** 31 - 1)


@pytest.mark.parametrize("fused", [False, True])
def test_append_in_place(fused):
    check_append(65, 8, 2, 128, 16, BF16, 128, False, "none", 1.0, False, fused, 5, in_place=True)


def test_append_without_rope_copies_bits():
    gen = torch.Generator(device=DEV).manual_seed(1)
    pool, k_pool, v_pool = make_pool(9, 16, 3, 64, F16)
    x = rand(gen, 50, 7, 64, dtype=F16)
    x[3] = math.nan
    k, v = x[:, 1:4], x[:, 4:]
    slots = random.Random(2).sample(range(9 * 16), 50)
    slots[7] = -9
    pkv.kv_append_tokens(pool, k, v, i64(slots))
    for got, src, fill in ((k_pool, k, 7.0), (v_pool, v, -7.0)):
        want = torch.full((9 * 16, 3, 64), fill, dtype=F16)
        for i, s in enumerate(slots):
            if s >= 0:
                want[s] = src[i].cpu()
        flat = got.transpose(1, 2).reshape(9 * 16, 3, 64).cpu()
        assert torch.equal(flat.view(torch.int16), want.view(torch.int16))


def test_append_keys_only_and_bad_slots():
    gen = torch.Generator(device=DEV).manual_seed(1)
    pool, k_pool, v_pool = make_pool(4, 16, 2, 64, BF16)
    k, v = rand(gen, 3, 2, 64, dtype=BF16), rand(gen, 3, 2, 64, dtype=BF16)
    st = status_word()
    pkv.kv_append_tokens(pool, k, v, i64([5, 64, 2 ** 40]), positions=i32([9, 9, 9]),
                         rope=pkv.Rope(64), dev_status=st)
    assert st.item() == ref.BAD_PAGE
    want, err = ref.turned(k[:1], torch.tensor([9]), ref.frequencies(64, 10000.0), False)
    ref.close(k_pool[0, :, 5][None], want, ref.rounded(want, err, BF16))
    v_pool[0, :, 5] = -7.0
    k_pool[0, :, 5] = 7.0
    assert (v_pool == -7.0).all() and (k_pool == 7.0).all()


def test_append_binding_refusals():
    pool, _, _ = make_pool(4, 16, 2, 64, BF16)
    k = torch.zeros(3, 2, 64, dtype=BF16, device=DEV)
    s, p = i64([0, 1, 2]), i32([0, 1, 2])
    rope = pkv.Rope(64)
    bad = [dict(k_new=k.half()), dict(k_new=k[:2]), dict(k_new=k.cpu()), dict(slots=s.int()),
           dict(k_new=k.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(v_new=torch.zeros(3, 3, 64, dtype=BF16, device=DEV)), dict(q=k), dict(positions=p),
           dict(rope=rope), dict(rope=rope, positions=p, q=k), dict(rope=rope, positions=s),
           dict(rope=rope, positions=p[:2]), dict(k_norm_weight=k[0, 0]),
           dict(rope=rope, positions=p, q_norm_weight=k[0, 0]),
           dict(rope=rope, positions=p, k_norm_weight=k[0, 0, :32])]
    for kw in bad:
        a = dict(k_new=k, v_new=k, slots=s)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            pkv.kv_append_tokens(pool, **a)


# ---------------------------------------------------------------------------
# bounds
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d,hkv,page,dtype", [(64, 2, 16, F16), (128, 8, 16, BF16),
                                              (128, 1, 48, F16), (64, 3, 256, BF16)])
@pytest.mark.parametrize("tokens", [1, 5, 64, 3000])
def test_bounds(d, hkv, page, dtype, tokens):
    gen = torch.Generator(device=DEV).manual_seed(tokens)
    rng = random.Random(tokens)
    NP = 2 * tokens + 5
    k_pool = rand(gen, NP, hkv, page, d, dtype=dtype)
    k_pool[::7] = 0.0
    pool = pkv.kv_pool_create(NP, page, hkv, d, dtype, k_pool, torch.empty_like(k_pool))
    # runs of consecutive slots on pages of their own, padding among them
    ids, slots = rng.sample(range(NP), tokens), []
    while len(slots) < tokens:
        first = rng.randrange(page)
        n = rng.choice([1, 1, page - first])
        pg = ids.pop()
        slots += [pg * page + first + i for i in range(n)]
        slots += [-1] * rng.choice([0, 0, 1])
    slots = slots[:tokens]
    bounds = torch.full((NP, hkv, 2, d), 55.0, dtype=dtype, device=DEV)
    want = ref.page_bounds(k_pool.cpu(), slots, bounds.cpu(), page)
    # rows behind a run are not read
    for s in slots:
        if s >= 0 and s + 1 not in slots and s % page + 1 < page:
            k_pool[s // page, :, s % page + 1:] = math.nan
    st = status_word()
    pkv.kv_page_bounds(pool, i64(slots), bounds, dev_status=st)
    assert torch.equal(bounds.cpu(), want) and st.item() == 0


def test_bounds_of_nan_inf_and_bad_slots():
    k_pool = torch.zeros(4, 1, 16, 64, dtype=BF16, device=DEV)
    k_pool[1, 0, 3, 5] = math.nan
    k_pool[2, 0, 0, 6] = math.inf
    k_pool[2, 0, 1, 7] = -math.inf
    pool = pkv.kv_pool_create(4, 16, 1, 64, BF16, k_pool, torch.empty_like(k_pool))
    bounds = torch.full((4, 1, 2, 64), 9.0, dtype=BF16, device=DEV)
    st = status_word()
    pkv.kv_page_bounds(pool, i64([19, 33, 33, 64, -1, 2 ** 40]), bounds, dev_status=st)
    assert st.item() == ref.BAD_PAGE
    want = torch.full((4, 1, 2, 64), 9.0, dtype=BF16)
    want[1:3] = 0.0
    want[1, 0, :, 5] = math.nan
    want[2, 0, 1, 6], want[2, 0, 0, 7] = math.inf, -math.inf
    assert torch.allclose(bounds.cpu().float(), want.float(), rtol=0, atol=0, equal_nan=True)


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------
def run_select(q, bounds, table, lens, page, keep, first, last, status=None, stream=None):
    B, Hkv = q.shape[0], bounds.shape[1]
    sel = torch.full((B, Hkv, keep), 77, dtype=torch.int32, device=DEV)
    ws = pkv.alloc_select_workspace(B, Hkv, table.shape[1])
    ws.fill_(255)
    pkv.paged_select_pages(q, bounds, table, lens, page, sel, ws, keep_first=first,
                           keep_last=last, dev_status=status, stream=stream)
    return sel


def check_select(q, bounds, table, lens, page, keep, first, last):
    st = status_word()
    got = run_select(q, bounds, i32(table), i32(lens), page, keep, first, last, st)
    want, flags = ref.select(q, bounds, table, lens, page, keep, first, last)
    assert got.tolist() == want
    assert st.item() == flags
    return flags


def page_table(rng, lens, page, NP, cols):
    ids = rng.sample(range(NP), sum(-(-n // page) for n in lens))
    table = []
    for n in lens:
        k = -(-n // page)
        table.append([ids.pop() for _ in range(k)] + [-1] * (cols - k))
    return table


@pytest.mark.parametrize("hq,hkv,d,page,dtype,keep,first,last,lens", [
    (4, 2, 64, 16, F16, 8, 1, 2, [300, 1000]),
    (32, 8, 128, 16, BF16, 16, 1, 1, [0, 1, 16, 255, 256, 257, 4000]),
    (28, 4, 128, 32, F16, 5, 0, 0, [161, 160, 3000]),
    (20, 1, 64, 48, BF16, 7, 3, 4, [48 * 7, 48 * 7 + 1, 9000]),
    (3, 3, 128, 256, BF16, 9, 0, 8, [256 * 9 + 1, 256 * 40]),
    (40, 2, 128, 16, F16, 1, 0, 0, [17, 500, 16]),
    (8, 2, 64, 16, BF16, 130, 2, 2, [16 * 131, 16 * 1000 - 3]),
])
def test_select(hq, hkv, d, page, dtype, keep, first, last, lens):
    gen = torch.Generator(device=DEV).manual_seed(hq)
    rng = random.Random(hq)
    NP = sum(-(-n // page) for n in lens) + 3
    cols = max(-(-n // page) for n in lens) + 2
    mid = rand(gen, NP, hkv, 1, d, dtype=torch.float32)
    half = torch.rand(NP, hkv, 1, d, generator=gen, device=DEV)
    bounds = torch.cat([mid - half, mid + half], 2).to(dtype)
    check_select(rand(gen, len(lens), hq, d, dtype=dtype), bounds,
                 page_table(rng, lens, page, NP, cols), lens, page, keep, first, last)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [400, 5000])
def test_select_scores_that_32_bits_cannot_tell_apart(dtype, n):
    """Scores of about 2000 that differ by multiples of 2^-14: below a step of fp32 there
    (2^-13), exact in 64 bits."""
    rng = random.Random(n)
    bounds = torch.full((n + 2, 1, 2, 64), 8.0, dtype=dtype)
    q = torch.full((1, 2, 64), 4.0, dtype=dtype)
    q[:, 1] = 0.0
    q[0, 0, 17] = 2.0 ** -7
    for p in range(n + 2):
        bounds[p, 0, :, 17] = rng.randrange(0, 60) * 2.0 ** -7
    table = page_table(rng, [16 * n], 16, n + 2, n)
    check_select(q.to(DEV), bounds.to(DEV), table, [16 * n], 16, 37, 1, 1)
    check_select(-q.to(DEV), -bounds.to(DEV), table, [16 * n], 16, 37, 1, 1)


@pytest.mark.parametrize("n,keep", [(40, 8), (300, 9), (3000, 1000)])
def test_select_equal_scores_take_the_lowest_index(n, keep):
    gen = torch.Generator(device=DEV).manual_seed(n)
    rng = random.Random(n)
    q = rand(gen, 2, 4, 64, dtype=BF16)
    table = page_table(rng, [16 * n, 16 * n - 7], 16, 2 * n, n)
    lens = [16 * n, 16 * n - 7]
    one = rand(gen, 1, 2, 2, 64, dtype=BF16).expand(2 * n, 2, 2, 64).contiguous()
    check_select(q, one, table, lens, 16, keep, 1, 1)          # all pages alike
    two = one.clone()
    two[::3] += 0.5                                            # two kinds of pages
    check_select(q, two, table, lens, 16, keep, 1, 1)
    check_select(torch.zeros_like(q), two, table, lens, 16, keep, 0, 1)  # all scores 0
    check_select(q, torch.zeros_like(two), table, lens, 16, keep, 1, 0)


def test_select_far_magnitudes():
    """bf16 values whose products leave fp32, in both directions."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    rng = random.Random(4)
    n = 200
    table = page_table(rng, [16 * n], 16, n, n)
    for big in (1e30, 1e-30):
        q = rand(gen, 1, 3, 64, dtype=BF16) * big
        bounds = (rand(gen, n, 1, 2, 64, dtype=BF16) * big).sort(2).values
        check_select(q, bounds, table, [16 * n], 16, 20, 1, 1)


def test_select_nan_and_inf():
    gen = torch.Generator(device=DEV).manual_seed(4)
    rng = random.Random(4)
    n = 150
    table = page_table(rng, [16 * n], 16, n, n)
    q = rand(gen, 1, 2, 64, dtype=F16)
    bounds = rand(gen, n, 1, 2, 64, dtype=F16).sort(2).values
    for p, x in ((40, math.nan), (90, math.nan), (60, math.inf)):
        bounds[table[0][p], 0, 1, 9] = x
    check_select(q, bounds, table, [16 * n], 16, 12, 1, 1)
    q[0, 1, 3] = math.nan                                      # every score NaN
    check_select(q, bounds, table, [16 * n], 16, 12, 1, 1)


def test_select_bad_pages_and_lengths():
    gen = torch.Generator(device=DEV).manual_seed(4)
    rng = random.Random(4)
    n = 60
    table = page_table(rng, [16 * n] * 4, 16, 4 * n, n)
    table[0][7], table[0][20], table[1][3] = -1, 4 * n, 2 ** 31 - 1
    for j in range(2, n):
        table[2][j] = -3                                       # not enough good pages
    q = rand(gen, 4, 4, 128, dtype=BF16)
    bounds = rand(gen, 4 * n, 2, 2, 128, dtype=BF16).sort(2).values
    flags = check_select(q, bounds, table, [16 * n, 16 * n - 1, 16 * n, 16 * n + 1], 16, 12, 1, 1)
    assert flags == ref.BAD_PAGE | ref.BAD_LEN
    assert check_select(q, bounds, table, [-1, 0, 5, 30], 16, 12, 1, 1) == ref.BAD_LEN


def test_select_many_pages():
    """More pages than the chosen ones' words of one round of the CTA, and a table of the
    largest width."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    rng = random.Random(9)
    n = 40000
    bounds = rand(gen, n, 1, 2, 64, dtype=F16).sort(2).values
    table = page_table(rng, [16 * n], 16, n, 131072)
    check_select(rand(gen, 1, 1, 64, dtype=F16), bounds, table, [16 * n], 16, 300, 1, 1)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def run_attend(q, k_pool, v_pool, table, lens, sel, scale, status=None, stream=None):
    out = torch.full_like(q, 5.0)
    pkv.paged_decode_attention_selected(q, k_pool, v_pool, table, lens, sel, scale, out,
                                        dev_status=status, stream=stream)
    return out


def check_attend(q, k_pool, v_pool, table, lens, sel, scale, flags=0):
    st = status_word()
    got = run_attend(q, k_pool, v_pool, i32(table), i32(lens), i32(sel), scale, st)
    want, bound = ref.attend(q, k_pool, v_pool, table, lens, sel, scale)
    ref.close(got, want, bound)
    assert st.item() == flags
    return got


def some_lists(rng, lens, hkv, page, keep):
    res = []
    for n in lens:
        pages = -(-n // page)
        res.append([])
        for _ in range(hkv):
            take = sorted(rng.sample(range(pages), min(pages, rng.choice([keep, keep, keep // 2]))))
            res[-1].append(take + [-1] * (keep - len(take)))
    return res


@pytest.mark.parametrize("hq,hkv,d,page,dtype,keep,lens", [
    (4, 2, 64, 16, F16, 8, [37, 100]),
    (1, 1, 128, 16, BF16, 1, [1]),
    (32, 8, 128, 16, BF16, 40, [0, 1, 15, 16, 17, 3000, 640]),
    (28, 4, 128, 32, F16, 20, [161, 5000, 31]),
    (20, 1, 64, 48, BF16, 7, [9000, 49, 200]),
    (9, 1, 128, 16, F16, 70, [2000, 3]),
    (16, 1, 128, 64, BF16, 9, [1000]),
    (34, 2, 64, 16, F16, 33, [900, 100]),
    (6, 3, 128, 256, BF16, 6, [256 * 9 + 1, 256 * 4, 255]),
    (4, 4, 64, 16, BF16, 300, [16 * 400 - 5]),
])
def test_attend(hq, hkv, d, page, dtype, keep, lens):
    gen = torch.Generator(device=DEV).manual_seed(hq)
    rng = random.Random(hq)
    NP = sum(-(-n // page) for n in lens) + 2
    cols = max(-(-n // page) for n in lens) + 1
    table = page_table(rng, lens, page, NP, cols)
    k_pool = rand(gen, NP, hkv, page, d, dtype=dtype)
    v_pool = rand(gen, NP, hkv, page, d, dtype=dtype)
    for b, n in enumerate(lens):  # what lies behind a sequence's end is never used
        if n % page:
            k_pool[table[b][n // page], :, n % page:] = math.nan
            v_pool[table[b][n // page], :, n % page:] = math.nan
    q = rand(gen, len(lens), hq, d, dtype=dtype)
    sel = some_lists(rng, lens, hkv, page, keep)
    got = check_attend(q, k_pool, v_pool, table, lens, sel, d ** -0.5)
    again = run_attend(q, k_pool, v_pool, i32(table), i32(lens), i32(sel), d ** -0.5)
    assert torch.equal(got, again)


def test_attend_many_requests():
    """Enough units that a cluster is a single CTA."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    rng = random.Random(1)
    lens = [rng.randrange(0, 400) for _ in range(80)]
    table = page_table(rng, lens, 16, 2100, 25)
    k_pool, v_pool = (rand(gen, 2100, 4, 16, 128, dtype=BF16) for _ in range(2))
    q = rand(gen, 80, 12, 128, dtype=BF16)
    check_attend(q, k_pool, v_pool, table, lens, some_lists(rng, lens, 4, 16, 12), 0.09)


def test_attend_all_pages_is_the_plain_decode():
    gen = torch.Generator(device=DEV).manual_seed(2)
    rng = random.Random(2)
    lens = [100, 1, 777, 2048]
    table = page_table(rng, lens, 16, 300, 128)
    k_pool, v_pool = (rand(gen, 300, 2, 16, 128, dtype=BF16) for _ in range(2))
    q = rand(gen, 4, 8, 128, dtype=BF16)
    sel = [[list(range(-(-n // 16))) + [-1] * (128 - -(-n // 16))] * 2 for n in lens]
    got = check_attend(q, k_pool, v_pool, table, lens, sel, 0.1)
    ws = pkv.alloc_workspace(4, 8, 2, 128)
    plain = torch.empty_like(q)
    pkv.paged_decode_attention(q, k_pool, v_pool, i32(table), i32(lens), 0.1, plain, ws)
    _, bound = ref.attend(q, k_pool, v_pool, table, lens, sel, 0.1)
    assert ((got.double() - plain.double()).abs().cpu() <= 2 * bound).all()


@pytest.mark.parametrize("case,flags", [
    ("holes", 0), ("twice", ref.BAD_LEN), ("descending", ref.BAD_LEN), ("beyond", ref.BAD_LEN),
    ("no page", ref.BAD_PAGE), ("length", ref.BAD_LEN), ("negative length", ref.BAD_LEN),
    ("all holes", 0), ("all bad", ref.BAD_PAGE)])
def test_attend_lists_and_data_that_are_off(case, flags):
    gen = torch.Generator(device=DEV).manual_seed(3)
    rng = random.Random(3)
    lens = [200, 150]
    table = page_table(rng, lens, 16, 40, 14)
    k_pool, v_pool = (rand(gen, 40, 2, 16, 64, dtype=F16) for _ in range(2))
    q = rand(gen, 2, 4, 64, dtype=F16)
    sel = some_lists(rng, lens, 2, 16, 6)
    if case == "holes":
        sel[0][1] = [-1, 3, -7, 5, -1, 12]
    elif case == "twice":
        sel[1][0] = [2, 2, 5, 5, 5, 8]
    elif case == "descending":
        sel[1][0] = [8, 5, 6, 2, 1, 9]
    elif case == "beyond":
        sel[1][1] = [0, 9, 10, 13, 14, 2 ** 31 - 1]
    elif case == "no page":
        table[0][4], table[0][5] = 40, -1
        sel[0][0] = [3, 4, 5, 6, -1, -1]
    elif case == "length":
        lens[0] = 14 * 16 + 1
        table[0] = table[0][:13] + [table[0][0]]
        sel[0][0] = [10, 11, 12, 13, -1, -1]
    elif case == "negative length":
        lens[1] = -5
        sel[1] = [[-1] * 6] * 2
    elif case == "all holes":
        sel[0] = [[-1] * 6] * 2
    elif case == "all bad":
        table[0] = [-1] * 14
    check_attend(q, k_pool, v_pool, table, lens, sel, 0.125, flags)


def test_attend_nan_and_inf_in_use():
    """A NaN in a listed row gives NaN in that head's outputs, in a page not listed none."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    table = [[1, 2, 3, 4]]
    k_pool, v_pool = (rand(gen, 6, 2, 16, 64, dtype=BF16) for _ in range(2))
    k_pool[2, 0, 3, 5] = math.nan
    v_pool[4, 1, 0, 9] = math.nan
    k_pool[0] = v_pool[5] = math.nan
    q = rand(gen, 1, 4, 64, dtype=BF16)
    sel = [[[0, 2, 3], [0, 1, 2]]]
    check_attend(q, k_pool, v_pool, table, [64], sel, 0.125)
    got = run_attend(q, k_pool, v_pool, i32(table), i32([64]), i32([[[0, 1, 3], [0, 2, 3]]]), 0.125)
    assert got[0, :2].isnan().all()
    assert got[0, 2:, 9].isnan().all() and not got[0, 2:, :9].isnan().any()


@pytest.mark.parametrize("scale", [0.0, -0.3, 30.0])
def test_attend_scales(scale):
    gen = torch.Generator(device=DEV).manual_seed(3)
    rng = random.Random(3)
    table = page_table(rng, [300], 16, 30, 20)
    k_pool, v_pool = (rand(gen, 30, 1, 16, 128, dtype=BF16) for _ in range(2))
    check_attend(rand(gen, 1, 3, 128, dtype=BF16), k_pool, v_pool, table, [300],
                 some_lists(rng, [300], 1, 16, 12), scale)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Server:
    """The state of a batch that is served with selected pages: fixed buffers, so that a
    step can be captured."""

    def __init__(self, batch, hq, hkv, d, page, dtype, cols, keep, tokens, seed, num_pages=400):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.gen, self.page, self.scale = g, page, d ** -0.5
        self.shape = (batch, hq, hkv, d, dtype)
        self.k, self.v = (torch.full((num_pages, hkv, page, d), math.nan, dtype=dtype, device=DEV)
                          for _ in range(2))
        self.pool = pkv.kv_pool_create(num_pages, page, hkv, d, dtype, self.k, self.v)
        self.free = i32(random.Random(seed).sample(range(num_pages), num_pages))
        self.begin, self.end = i32([0]), i32([0])
        self.cached, self.new, self.lens = (i32([0] * batch) for _ in range(3))
        self.starts = i32([0] * (batch + 1))
        self.table = torch.full((batch, cols), -1, dtype=torch.int32, device=DEV)
        self.bounds = torch.full((num_pages, hkv, 2, d), math.nan, dtype=dtype, device=DEV)
        self.rope = pkv.Rope(d, 10000.0, scaling="turns", factor=4.0, original_context=64.0)
        self.sel = torch.full((batch, hkv, keep), -1, dtype=torch.int32, device=DEV)
        self.ws = pkv.alloc_select_workspace(batch, hkv, cols)
        self.status = status_word()
        self.history = [[] for _ in range(batch)]  # (k, v) rows as given, for the plain form
        self.resize(tokens)

    def resize(self, tokens):
        B, hq, hkv, d, dt = self.shape
        self.pos, self.seq = i32([0] * tokens), i32([0] * tokens)
        self.slots = i64([0] * tokens)
        self.x = torch.zeros(tokens, hq + 2 * hkv, d, dtype=dt, device=DEV)
        self.q_rot = torch.zeros(tokens, hq, d, dtype=dt, device=DEV)
        self.q_last = torch.zeros(B, hq, d, dtype=dt, device=DEV)
        self.out = torch.zeros(B, hq, d, dtype=dt, device=DEV)

    def step(self, stream=None):
        _, hq, hkv, _, _ = self.shape
        q, k, v = self.x.split([hq, hkv, hkv], 1)
        pkv.paged_tables_build(self.cached, self.new, self.free, self.begin, self.end, self.table,
                               self.page, self.k.shape[0], self.lens, self.starts, self.pos,
                               self.seq, self.slots, dev_status=self.status)
        pkv.kv_append_tokens(self.pool, k, v, self.slots, q=q, positions=self.pos, rope=self.rope,
                             q_out=self.q_rot, dev_status=self.status)
        pkv.kv_page_bounds(self.pool, self.slots, self.bounds, dev_status=self.status)
        # each request's last token asks
        torch.index_select(self.q_rot, 0, (self.starts[1:] - 1).clamp(min=0), out=self.q_last)
        pkv.paged_select_pages(self.q_last, self.bounds, self.table, self.lens, self.page,
                               self.sel, self.ws, keep_first=1, keep_last=2,
                               dev_status=self.status)
        pkv.paged_decode_attention_selected(self.q_last, self.k, self.v, self.table, self.lens,
                                            self.sel, self.scale, self.out,
                                            dev_status=self.status)

    def feed(self, new):
        """New tokens' projections and lengths for the next step."""
        self.x.copy_(torch.randn(self.x.shape, generator=self.gen, device=DEV).to(self.x.dtype))
        self.new.copy_(i32(new))

    def check(self):
        """The step's outputs against the parts' plain forms on what is in the cache."""
        assert self.status.item() == 0
        lens, table = self.lens.tolist(), self.table.tolist()
        flat = [t for row, n in zip(table, lens) for t in row[:-(-n // self.page)]]
        assert len(flat) == len(set(flat)) and min(flat, default=0) >= 0
        assert self.slots.tolist() == [
            -1 if s < 0 else table[s][p // self.page] * self.page + p % self.page
            for s, p in zip(self.seq.tolist(), self.pos.tolist())]
        for row, n in zip(table, lens):
            for j in range(-(-n // self.page)):
                rows = self.k[row[j], :, :min(self.page, n - j * self.page)]
                assert torch.equal(self.bounds[row[j], :, 0], rows.amin(1))
                assert torch.equal(self.bounds[row[j], :, 1], rows.amax(1))
        want, _ = ref.select(self.q_last, self.bounds, table, lens, self.page, self.sel.shape[2],
                             1, 2)
        assert self.sel.tolist() == want
        out, bound = ref.attend(self.q_last, self.k, self.v, table, lens, want, self.scale)
        ref.close(self.out, out, bound)
        # the cached keys are the given ones, turned at their positions
        _, hq, hkv, _, dt = self.shape
        k = self.x[:, hq:hq + hkv]
        live = self.pos >= 0
        y, err = ref.turned(k[live], self.pos[live],
                            ref.frequencies(k.shape[2], 10000.0, "turns", 4.0, context=64.0), False)
        s = self.slots[live]
        got = self.k[s // self.page, :, s % self.page]
        ref.close(got, y, ref.rounded(y, err, dt))
        assert torch.equal(self.v[s // self.page, :, s % self.page], self.x[live][:, hq + hkv:])

    def advance(self):
        self.cached.copy_(self.lens)
        self.begin.copy_(self.end)


@pytest.mark.parametrize("dtype,hq,hkv,d,page", [(BF16, 8, 2, 128, 16), (F16, 6, 1, 64, 32)])
def test_prompts_then_steps(dtype, hq, hkv, d, page):
    s = Server(5, hq, hkv, d, page, dtype, cols=40, keep=6, tokens=700, seed=1)
    s.feed([200, 1, 0, 333, 47])
    s.step()
    s.check()
    s.advance()
    s.resize(40)
    for i in range(20):
        s.feed([1, 1, i % 2, 1, 1 if i < 18 else 0])
        s.step()
        s.check()
        s.advance()
    s.resize(200)                       # a late prompt beside requests that decode
    s.feed([1, 120, 1, 1, 9])
    s.step()
    s.check()


def test_captured_step_replayed():
    s = Server(4, 8, 2, 128, 16, BF16, cols=30, keep=6, tokens=300, seed=2)
    s.feed([120, 90, 3, 50])
    s.step()
    s.check()
    s.advance()
    s.resize(4)
    s.feed([1, 1, 1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    torch.cuda.current_stream().wait_stream(side)
    s.check()
    s.advance()                         # (the warm-up's tokens are the requests' own)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for i in range(12):
        s.feed([1, int(i % 3 > 0), 1, 1])
        graph.replay()
        s.check()
        s.advance()


def test_calls_on_another_stream():
    """Given a stream, a call runs on it, not on the current one."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    rng = random.Random(1)
    lens = [500]
    table = page_table(rng, lens, 16, 40, 32)
    k_pool, v_pool = (rand(gen, 40, 2, 16, 64, dtype=BF16) for _ in range(2))
    q, bounds = rand(gen, 1, 4, 64, dtype=BF16), rand(gen, 40, 2, 2, 64, dtype=BF16).sort(2).values
    t, n = i32(table), i32(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sel = run_select(q, bounds, t, n, 16, 8, 1, 1, stream=side)
    out = torch.empty_like(q)
    side.wait_stream(torch.cuda.current_stream())
    pkv.paged_decode_attention_selected(q, k_pool, v_pool, t, n, sel, 0.1, out, stream=side)
    side.synchronize()
    want, _ = ref.select(q, bounds, table, lens, 16, 8, 1, 1)
    assert sel.tolist() == want
    w, b = ref.attend(q, k_pool, v_pool, table, lens, want, 0.1)
    ref.close(out, w, b)


def test_binding_refusals():
    q = torch.zeros(2, 4, 64, dtype=BF16, device=DEV)
    kp = torch.zeros(4, 2, 16, 64, dtype=BF16, device=DEV)
    bounds = torch.zeros(4, 2, 2, 64, dtype=BF16, device=DEV)
    t, n = i32([[0, 1], [2, 3]]), i32([5, 20])
    sel = torch.zeros(2, 2, 3, dtype=torch.int32, device=DEV)
    ws = pkv.alloc_select_workspace(2, 2, 2)
    out = torch.empty_like(q)
    good = dict(q=q, bounds=bounds, page_table=t, context_lens=n, page_size=16, selected=sel,
                workspace=ws)
    pkv.paged_select_pages(**good)
    for kw in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[:1]), dict(bounds=bounds[:, :1]),
               dict(bounds=bounds.transpose(0, 1)), dict(page_table=t.long()),
               dict(context_lens=n[:1]), dict(selected=sel[:, :1].contiguous()),
               dict(selected=sel.long()), dict(workspace=ws.int()), dict(q=None)):
        with pytest.raises((ValueError, TypeError)):
            pkv.paged_select_pages(**dict(good, **kw))
    with pytest.raises(pkv.PagedKVError, match="WORKSPACE"):
        pkv.paged_select_pages(**dict(good, workspace=ws[:16]))
    good = dict(q=q, k_pool=kp, v_pool=kp, page_table=t, context_lens=n, selected=sel, scale=1.0,
                out=out)
    pkv.paged_decode_attention_selected(**good)
    for kw in (dict(q=q.half()), dict(k_pool=kp.half()), dict(v_pool=kp[:2]), dict(out=out[:1]),
               dict(out=out.transpose(0, 1)), dict(selected=sel[:1]), dict(page_table=t[:1]),
               dict(k_pool=kp.cpu())):
        with pytest.raises((ValueError, TypeError)):
            pkv.paged_decode_attention_selected(**dict(good, **kw))
    with pytest.raises(pkv.PagedKVError, match="ALIAS"):
        pkv.paged_decode_attention_selected(**dict(good, out=q))
    e = i32([0])
    good = dict(cached_lens=n, new_lens=n, free_pages=i32([0, 1]), free_begin=None, free_end=e,
                page_table=t, page_size=16, num_pages=4, context_lens=i32([0, 0]),
                query_starts=i32([0, 0, 0]), positions=i32([0] * 4), seq_ids=i32([0] * 4),
                slots=i64([0] * 4))
    pkv.paged_tables_build(**good)
    for kw in (dict(new_lens=n[:1]), dict(free_end=i32([0, 0])), dict(query_starts=i32([0, 0])),
               dict(slots=i32([0] * 4)), dict(positions=i32([0] * 3)), dict(page_table=t[0]),
               dict(cached_lens=n.cpu()), dict(free_begin=n)):
        with pytest.raises((ValueError, TypeError)):
            pkv.paged_tables_build(**dict(good, **kw))


# ---------------------------------------------------------------------------
# the ends of the ranges
# ---------------------------------------------------------------------------
def test_offsets_beyond_32_bits():
    """A pool of 2.4e9 elements a side: rows of its last pages are written, bounded,
    selected and attended to at their own places."""
    NP, hkv, page, d = 9200, 8, 256, 128
    assert NP * hkv * page * d > 2 ** 31
    gen = torch.Generator(device=DEV).manual_seed(6)
    k_pool = torch.empty(NP, hkv, page, d, dtype=BF16, device=DEV)
    v_pool = torch.empty_like(k_pool)
    pool = pkv.kv_pool_create(NP, page, hkv, d, BF16, k_pool, v_pool)
    table = [[NP - 1, 3, NP - 2, NP - 5, NP - 9]]
    n = 4 * page + 100
    slots = [table[0][t // page] * page + t % page for t in range(n)]
    k, v = rand(gen, n, hkv, d, dtype=BF16), rand(gen, n, hkv, d, dtype=BF16)
    q = rand(gen, n, 16, d, dtype=BF16)
    q_out = torch.empty_like(q)
    st = status_word()
    pkv.kv_append_tokens(pool, k, v, i64(slots), q=q, positions=i32(list(range(n))),
                         rope=pkv.Rope(d), q_out=q_out, dev_status=st)
    want, err = ref.turned(k, torch.arange(n), ref.frequencies(d, 10000.0), False)
    at = torch.tensor(slots)
    got = k_pool[at // page, :, at % page]
    ref.close(got, want, ref.rounded(want, err, BF16))
    assert torch.equal(v_pool[at // page, :, at % page], v)
    bounds = torch.zeros(NP, hkv, 2, d, dtype=BF16, device=DEV)
    pkv.kv_page_bounds(pool, i64(slots), bounds, dev_status=st)
    for j, p in enumerate(table[0]):
        rows = k_pool[p, :, :min(page, n - j * page)]
        assert torch.equal(bounds[p, :, 0], rows.amin(1))
        assert torch.equal(bounds[p, :, 1], rows.amax(1))
    ask = q_out[-1:]
    sel = run_select(ask, bounds, i32(table), i32([n]), page, 3, 0, 1, st)
    lists, _ = ref.select(ask, bounds, table, [n], page, 3, 0, 1)
    assert sel.tolist() == lists
    out = run_attend(ask, k_pool, v_pool, i32(table), i32([n]), sel, 0.09, st)
    small = [[0, 1, 2, 3, 4]]  # the same pages in a small pool for the plain form
    w, b = ref.attend(ask, k_pool[table[0]], v_pool[table[0]], small, [n], lists, 0.09)
    ref.close(out, w, b)
    assert st.item() == 0


def test_append_many_tokens_and_rows():
    """Several groups a CTA, and tokens of more rows than a group's."""
    check_append(9001, 8, 2, 128, 16, BF16, 128, False, "none", 1.0, True, True, 21)
    check_append(3, 900, 62, 64, 16, F16, 32, True, "none", 1.0, False, False, 22)
    check_append(2, 2000, 1000, 64, 16, F16, 64, False, "none", 1.0, False, False, 23)


def test_append_norm_of_one_side():
    gen = torch.Generator(device=DEV).manual_seed(4)
    q, k, v = token_rows(gen, 20, 6, 2, 128, F16, True)
    w = (1 + 0.2 * rand(gen, 128, dtype=torch.float32)).half()
    pos = list(range(5, 25))
    for qw, kw in ((w, None), (None, w)):
        pool, k_pool, _ = make_pool(2, 16, 2, 128, F16)
        q_out = torch.empty(20, 6, 128, dtype=F16, device=DEV)
        pkv.kv_append_tokens(pool, k, v, i64(list(range(20))), q=q, positions=i32(pos),
                             rope=pkv.Rope(64), q_out=q_out, q_norm_weight=qw, k_norm_weight=kw,
                             norm_eps=1e-5)
        f = ref.frequencies(64, 10000.0)
        for got, x, weight in ((q_out, q, qw),
                               (k_pool.transpose(1, 2).reshape(32, 2, 128)[:20], k, kw)):
            y, err = ref.turned(x, torch.tensor(pos), f, False, 1.0, weight, 1e-5)
            ref.close(got, y, ref.rounded(y, err, F16))


def test_append_one_slot_twice():
    gen = torch.Generator(device=DEV).manual_seed(4)
    pool, k_pool, v_pool = make_pool(1, 16, 1, 64, F16)
    k, v = rand(gen, 2, 1, 64, dtype=F16), rand(gen, 2, 1, 64, dtype=F16)
    pkv.kv_append_tokens(pool, k, v, i64([3, 3]))
    vecs = k_pool[0, 0, 3].reshape(8, 8)
    assert all(torch.equal(vecs[i], k[0, 0].reshape(8, 8)[i])
               or torch.equal(vecs[i], k[1, 0].reshape(8, 8)[i]) for i in range(8))
    v_pool[0, 0, 3] = -7.0
    assert (v_pool == -7.0).all()


def test_calls_with_no_tokens_or_requests():
    pool, k_pool, v_pool = make_pool(4, 16, 2, 64, BF16)
    k = torch.empty(0, 2, 64, dtype=BF16, device=DEV)
    none = i64([])
    pkv.kv_append_tokens(pool, k, k, none)
    q = torch.empty(0, 4, 64, dtype=BF16, device=DEV)
    pkv.kv_append_tokens(pool, k, k, none, q=q, positions=i32([]), rope=pkv.Rope(64), q_out=q)
    pkv.kv_page_bounds(pool, none, torch.zeros(4, 2, 2, 64, dtype=BF16, device=DEV))
    t, n = i32([]).reshape(0, 3), i32([])
    sel = torch.empty(0, 2, 5, dtype=torch.int32, device=DEV)
    pkv.paged_select_pages(q, torch.zeros(4, 2, 2, 64, dtype=BF16, device=DEV), t, n, 16, sel,
                           pkv.alloc_select_workspace(0, 2, 3))
    pkv.paged_decode_attention_selected(q, k_pool, v_pool, t, n, sel, 0.1, torch.empty_like(q))
    torch.cuda.synchronize()
    assert (k_pool == 7.0).all() and (v_pool == -7.0).all()


def test_select_largest_group():
    gen = torch.Generator(device=DEV).manual_seed(8)
    rng = random.Random(8)
    bounds = rand(gen, 300, 1, 2, 128, dtype=BF16).sort(2).values
    table = page_table(rng, [16 * 300], 16, 300, 300)
    check_select(rand(gen, 1, 192, 128, dtype=BF16), bounds, table, [16 * 300], 16, 20, 1, 1)
    table = page_table(rng, [16 * 100], 16, 300, 100)
    check_select(rand(gen, 1, 192, 128, dtype=BF16), bounds, table, [16 * 100], 16, 20, 1, 1)


@pytest.mark.parametrize("cols", [40, 600, 2000])
def test_select_many_requests(cols):
    """Both forms of the selection over a whole grid of uneven requests."""
    gen = torch.Generator(device=DEV).manual_seed(cols)
    rng = random.Random(cols)
    lens = [rng.randrange(0, 16 * cols + 1) for _ in range(12)] + [16 * cols]
    NP = sum(-(-n // 16) for n in lens) + 2
    bounds = rand(gen, NP, 2, 2, 64, dtype=F16).sort(2).values
    check_select(rand(gen, 13, 8, 64, dtype=F16), bounds, page_table(rng, lens, 16, NP, cols),
                 lens, 16, 24, 1, 2)


@pytest.mark.parametrize("hq,hkv,d,page,dtype", [(8, 1, 128, 64, BF16), (12, 1, 64, 256, F16),
                                                 (16, 1, 128, 128, F16), (2, 1, 64, 64, BF16)])
def test_attend_of_few_units_over_clusters(hq, hkv, d, page, dtype):
    """Long lists of a single request: eight CTAs merge, also in a captured call."""
    gen = torch.Generator(device=DEV).manual_seed(hq)
    rng = random.Random(hq)
    n = page * 60 - 7
    table = page_table(rng, [n], page, 62, 64)
    k_pool, v_pool = (rand(gen, 62, hkv, page, d, dtype=dtype) for _ in range(2))
    q = rand(gen, 1, hq, d, dtype=dtype)
    sel = [[sorted(rng.sample(range(60), 50)) + [-1] * 3]]
    got = check_attend(q, k_pool, v_pool, table, [n], sel, d ** -0.5)
    t, ln, s, out = i32(table), i32([n]), i32(sel), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_decode_attention_selected(q, k_pool, v_pool, t, ln, s, d ** -0.5, out)
    graph.replay()
    assert torch.equal(out, got)
    short = [[rng.sample(range(60), 1) + [-1] * 52]]
    s.copy_(i32(short))
    graph.replay()
    w, b = ref.attend(q, k_pool, v_pool, table, [n], short, d ** -0.5)
    ref.close(out, w, b)


def test_attend_lists_that_are_mostly_empty():
    """A list as wide as the table, with its few entries far apart."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    k_pool, v_pool = (rand(gen, 40, 2, 16, 64, dtype=BF16) for _ in range(2))
    rng = random.Random(2)
    cols = 5000
    table = [[rng.randrange(40) for _ in range(cols)] for _ in range(2)]
    sel = [[[-1] * cols for _ in range(2)] for _ in range(2)]
    for b in range(2):
        for h in range(2):
            for j in rng.sample(range(cols), 3 * (b + h)):
                sel[b][h][j] = j
    q = rand(gen, 2, 8, 64, dtype=BF16)
    check_attend(q, k_pool, v_pool, table, [16 * cols, 16 * cols - 3], sel, 0.125)


def test_two_streams_at_once():
    """Calls with workspaces and outputs of their own on two streams."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    rng = random.Random(3)
    lens = [16 * 700, 16 * 650 - 5]
    table = page_table(rng, lens, 16, 1400, 700)
    bounds = rand(gen, 1400, 2, 2, 128, dtype=BF16).sort(2).values
    k_pool, v_pool = (rand(gen, 1400, 2, 16, 128, dtype=BF16) for _ in range(2))
    qs = [rand(gen, 2, 8, 128, dtype=BF16) for _ in range(2)]
    t, n = i32(table), i32(lens)
    want = [ref.select(q, bounds, table, lens, 16, 40, 1, 1)[0] for q in qs]
    sels = [torch.empty(2, 2, 40, dtype=torch.int32, device=DEV) for _ in range(2)]
    outs = [torch.empty_like(q) for q in qs]
    works = [pkv.alloc_select_workspace(2, 2, 700) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, q, sel, out, ws in zip(streams, qs, sels, outs, works):
            pkv.paged_select_pages(q, bounds, t, n, 16, sel, ws, stream=s)
            pkv.paged_decode_attention_selected(q, k_pool, v_pool, t, n, sel, 0.09, out, stream=s)
    torch.cuda.synchronize()
    for q, sel, out, lists in zip(qs, sels, outs, want):
        assert sel.tolist() == lists
        w, b = ref.attend(q, k_pool, v_pool, table, lens, lists, 0.09)
        ref.close(out, w, b)


def test_destroyed_pool_is_refused():
    pool, _, _ = make_pool(4, 16, 2, 64, BF16)
    pool.destroy()
    k = torch.zeros(1, 2, 64, dtype=BF16, device=DEV)
    with pytest.raises(ValueError, match="destroyed"):
        pkv.kv_append_tokens(pool, k, k, i64([0]))
    with pytest.raises(ValueError, match="destroyed"):
        pkv.kv_page_bounds(pool, i64([0]), torch.zeros(4, 2, 2, 64, dtype=BF16, device=DEV))


def test_pool_that_owns_its_memory():
    pool = pkv.kv_pool_create(4, 16, 2, 64, BF16)
    gen = torch.Generator(device=DEV).manual_seed(1)
    k, v = rand(gen, 20, 2, 64, dtype=BF16), rand(gen, 20, 2, 64, dtype=BF16)
    pkv.kv_append_tokens(pool, k, v, i64(list(range(20, 40))))
    got = [torch.zeros(1, 2, 40, 64, dtype=BF16, device=DEV) for _ in range(2)]
    pkv.kv_gather(pool, i32([[0, 1, 2]]), i32([40]), 40, *got)
    assert torch.equal(got[0][0, :, 20:], k.transpose(0, 1))
    assert torch.equal(got[1][0, :, 20:], v.transpose(0, 1))
    pool.destroy()


def test_selected_pool_of_8_bits_is_refused():
    pool = pkv.kv8_pool_create(4, 16, 2, 64)
    k = torch.zeros(1, 2, 64, dtype=BF16, device=DEV)
    with pytest.raises(ValueError, match="16-bit"):
        pkv.kv_append_tokens(pool, k, k, i64([0]))
    with pytest.raises(ValueError, match="16-bit"):
        pkv.kv_page_bounds(pool, i64([0]), torch.zeros(4, 2, 2, 64, dtype=BF16, device=DEV))

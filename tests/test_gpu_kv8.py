"""The 8-bit cache's operators against their plain 64-bit forms (kv8_ref).

Appended bytes are compared bit for bit where nothing is computed before the
rounding (no rotation, no norm).  Behind a rotation each stored value must be
within half an e4m3 step of the exact one, and outputs within
kv8_ref.attention_bound, whose parts are derived there."""
import numpy as np
import pytest
import torch

import kv8_ref as ref
import paged_kv_decode_16_gb300 as pkv

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DT = [torch.bfloat16, torch.float16]


class Cache:
    """A pool with random contents and a page table, on the GPU and in numpy."""

    def __init__(self, seed, lens, Hkv, D, P, exps=(-3, 3), extra=2, cap=None):
        rng = np.random.default_rng(seed)
        lens = np.asarray(lens)
        cap = lens if cap is None else np.asarray(cap)
        pages = [max(0, -(-int(n) // P)) for n in cap]
        NP = sum(pages) + extra
        perm = rng.permutation(NP)
        self.table = np.full((len(lens), max([1] + pages)), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        # contents: normal values to an amax near 448, as an append leaves them
        x = rng.standard_normal((2, NP, Hkv, P, D)) * 120
        self.k, self.v = ref.encode(x[0]), ref.encode(x[1])
        self.scales = (rng.integers(exps[0], exps[1] + 1, (NP, Hkv, P // 16, 2)) + 127).astype(
            np.uint8)
        # keys small enough for a softmax that is not one-hot
        self.scales[..., 0] = np.clip(self.scales[..., 0].astype(int), 118, 121)
        self.lens = lens.astype(np.int32)
        self.rng, self.D, self.P, self.Hkv, self.NP = rng, D, P, Hkv, NP

    def poison(self):
        """NaN in every row that no sequence attends to, and every byte of the
        scales of blocks that none does at random."""
        live = np.zeros((self.NP, self.P), dtype=bool)
        for b, n in enumerate(self.lens):
            for p in range(-(-int(n) // self.P)):
                live[self.table[b, p], :min(self.P, int(n) - p * self.P)] = True
        for pool in (self.k, self.v):
            pool[np.broadcast_to(~live[:, None, :, None], pool.shape)] = 0x7F
        dead = ~live.reshape(self.NP, 1, -1, 16).any(-1)
        dead = np.broadcast_to(dead[..., None], self.scales.shape)
        self.scales[dead] = self.rng.integers(0, 256, int(dead.sum()))
        return self

    def gpu(self):
        f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.k_g = f(self.k).view(torch.float8_e4m3fn)
        self.v_g = f(self.v).view(torch.float8_e4m3fn)
        self.s_g = f(self.scales).view(torch.float8_e8m0fnu)
        self.table_g, self.lens_g = f(self.table), f(self.lens)
        return self

    def pool(self):
        return pkv.kv8_pool_create(self.NP, self.P, self.Hkv, self.D, self.k_g, self.v_g, self.s_g)

    def back(self):
        return (self.k_g.view(torch.uint8).cpu().numpy(), self.v_g.view(torch.uint8).cpu().numpy(),
                self.s_g.view(torch.uint8).cpu().numpy())


def f64(t):
    return t.double().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def same_bytes(c, k, v, s, what=""):
    gk, gv, gs = c.back()
    assert np.array_equal(gs, s), f"{what}: scales"
    # the two NaN patterns are one value
    nan = lambda x: np.where((x & 0x7F) == 0x7F, 0x7F, x)  # noqa: E731
    assert np.array_equal(nan(gk), nan(k)), f"{what}: k"
    assert np.array_equal(nan(gv), nan(v)), f"{what}: v"


def new_rows(c, n, dtype, scale=1.0):
    size = c.rng.standard_normal((2, n, c.Hkv, c.D)) * scale * np.exp2(
        c.rng.integers(-3, 4, (2, n, c.Hkv, 1)))
    t = torch.from_numpy(size).to(dtype).cuda()
    return t[0].contiguous(), t[1].contiguous()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P,Hkv", [(128, 16, 2), (64, 32, 3), (128, 48, 1), (64, 256, 1)])
def test_append_token_by_token(dtype, D, P, Hkv):
    """Single tokens, one call each: blocks that fill up and change scale."""
    start = np.array([0, 5, 14, 31])
    c = Cache(1, start, Hkv, D, P, cap=start + 40).gpu()
    pool = c.pool()
    k, v, s = c.k.copy(), c.v.copy(), c.scales.copy()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(36):
        pos = start + step
        if step % 5 == 3:
            pos = pos.copy()
            pos[step % 4] = -1  # a padded slot
            start[step % 4] -= 1
        kn, vn = new_rows(c, 4, dtype)
        pkv.kv8_append(pool, kn, vn, c.table_g, i32(pos), dev_status=st)
        ref.append(k, v, s, f64(kn), f64(vn), c.table, pos, np.arange(4))
        if step % 7 == 0 or step == 35:
            same_bytes(c, k, v, s, f"step {step}")
    assert int(st) == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P,Hkv,start,count", [
    (128, 16, 2, [0, 0, 3, 15, 16, 1], [1, 16, 13, 17, 33, 0]),
    (64, 32, 1, [7, 0, 40], [200, 1, 30]),
    (128, 64, 4, [0], [1]),
    (64, 48, 2, [9] * 20, [1, 2, 3, 4, 5] * 4),
    (128, 16, 1, [0, 11, 0, 3], [700, 900, 601, 333]),  # more than 2048 tokens
    (64, 256, 2, [250, 1], [1100, 1500]),
])
def test_append_prompts(dtype, D, P, Hkv, start, count):
    start, count = np.array(start), np.array(count)
    c = Cache(2, start, Hkv, D, P, cap=start + count).gpu()
    seq = np.repeat(np.arange(len(count)), count)
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, count)])
    kn, vn = new_rows(c, len(pos), dtype)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.kv8_append(c.pool(), kn, vn, c.table_g, i32(pos), i32(seq), dev_status=st)
    k, v, s = c.k.copy(), c.v.copy(), c.scales.copy()
    ref.append(k, v, s, f64(kn), f64(vn), c.table, pos, seq)
    same_bytes(c, k, v, s)
    assert int(st) == 0


def test_append_order_of_sequences_and_gaps():
    """Tokens of different sequences in any order, skipped tokens between, and a
    sequence whose tokens come in two stretches of different blocks."""
    c = Cache(3, [64, 64, 64], 2, 128, 16).gpu()
    pos = np.array([32, 33, -1, 34, 5, 6, 7, 0, 1, -1, -1, 15, 16])
    seq = np.array([2, 2, 2, 0, 1, 1, 1, 2, 2, 0, 1, 0, 0])
    kn, vn = new_rows(c, len(pos), torch.bfloat16)
    pkv.kv8_append(c.pool(), kn, vn, c.table_g, i32(pos), i32(seq))
    k, v, s = c.k.copy(), c.v.copy(), c.scales.copy()
    ref.append(k, v, s, f64(kn), f64(vn), c.table, pos, seq)
    same_bytes(c, k, v, s)


def test_append_special_values():
    """Not finite -> NaN without a say in the scale; zeros; the scales' ends."""
    c = Cache(4, [16] * 8, 1, 64, 16).gpu()
    n = 8
    kn, vn = new_rows(c, n, torch.bfloat16)
    kn[0, 0, 3] = float("inf")
    kn[1, 0, 60] = float("nan")
    vn[2] = 0.0
    vn[3, 0, 0] = 3e38
    vn[4] = 1e-30
    vn[5] = float("-inf")
    vn[6, 0] = torch.linspace(-448.0, 448.0, 64)
    kn[7, 0, :] = 2.0 ** 40 * 448
    pos = np.zeros(n, dtype=np.int64)
    pkv.kv8_append(c.pool(), kn, vn, c.table_g, i32(pos))
    k, v, s = c.k.copy(), c.v.copy(), c.scales.copy()
    ref.append(k, v, s, f64(kn), f64(vn), c.table, pos, np.arange(n))
    same_bytes(c, k, v, s)
    # a later token in the same blocks: zero blocks grow, the others keep or grow
    kn, vn = new_rows(c, n, torch.float16)
    pkv.kv8_append(c.pool(), kn, vn, c.table_g, i32(pos + 1))
    ref.append(k, v, s, f64(kn), f64(vn), c.table, pos + 1, np.arange(n))
    same_bytes(c, k, v, s, "second token")


@pytest.mark.parametrize("single", [True, False])
def test_append_bad_inputs_leave_the_pool(single):
    c = Cache(5, [64] * 4, 2, 64, 16).gpu()
    before = [x.copy() for x in c.back()]
    c.table_g[1, 0] = c.NP
    c.table_g[2, 0] = -7
    kn, vn = new_rows(c, 4, torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = None if single else i32([0, 1, 2, 3])
    pkv.kv8_append(c.pool(), kn, vn, c.table_g, i32([64, 3, 4, 1 << 30]), seq, dev_status=st)
    assert int(st) == pkv.DEV_BAD_LEN | pkv.DEV_BAD_PAGE
    for a, b in zip(before, c.back()):
        assert np.array_equal(a, b)
    if not single:
        st.zero_()
        pkv.kv8_append(c.pool(), kn, vn, c.table_g, i32([0, 0, 0, 0]), i32([4, -1, 99, 1 << 30]),
                       dev_status=st)
        assert int(st) == pkv.DEV_BAD_SEQ
        # the same position twice, and a step back within a block: the later one is skipped
        st.zero_()
        pkv.kv8_append(c.pool(), kn, vn, c.table_g, i32([20, 20, 9, 8]), i32([0, 0, 3, 3]),
                       dev_status=st)
        assert int(st) == pkv.DEV_BAD_LEN
        k, v, s = before
        ref.append(k, v, s, f64(kn[::2]), f64(vn[::2]), c.table, np.array([20, 9]),
                   np.array([0, 3]))
        same_bytes(c, k, v, s)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,Hq,Hkv,theta,qn,kn_,big", [
    (128, 8, 2, 10000.0, False, False, 0), (64, 6, 2, 500000.0, True, True, 0),
    (128, 5, 1, 500000.0, False, True, 1 << 20), (64, 4, 4, 1e6, True, False, (1 << 31) - 4000),
])
def test_append_rope(dtype, D, Hq, Hkv, theta, qn, kn_, big):
    """The rotation (and norm): q_out rounded once, each stored key within half
    a step of the exact rotation.  `big`: far positions, from a page table whose
    far columns are the only ones in use."""
    P = 256 if big else 16
    count = np.array([40, 1, 23])
    start = np.array([3, 0, 16]) + big
    cap = start + count - big // P * P
    c = Cache(6, cap, Hkv, D, P).gpu()
    off = big // P
    table, table_g = c.table, c.table_g
    if big > 1 << 24:
        off = 0  # positions beyond any table: only q is rotated
    elif off:
        table_g = torch.zeros((3, off + table.shape[1]), dtype=torch.int32, device="cuda")
        table_g[:, off:] = c.table_g
    seq = np.repeat(np.arange(3), count)
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, count)])
    kn, vn = new_rows(c, len(pos), dtype)
    q = torch.randn(len(pos), Hq, D, dtype=torch.float64).to(dtype).cuda()
    wq = (1 + 0.2 * torch.randn(D)).to(dtype).cuda() if qn else None
    wk = (1 + 0.2 * torch.randn(D)).to(dtype).cuda() if kn_ else None
    out = torch.empty_like(q)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = q.clone()
    pkv.kv8_append_rope(c.pool(), q, kn, vn, table_g, i32(pos), theta, out, i32(seq),
                        dev_status=st, q_norm_weight=wq, k_norm_weight=wk, norm_eps=1e-5)
    assert torch.equal(q, keep)
    yq = ref.norm_rope(f64(q), None if wq is None else f64(wq), pos, theta, 1e-5)
    yk = ref.norm_rope(f64(kn), None if wk is None else f64(wk), pos, theta, 1e-5)
    # fp32: a few roundings of the norm, the products and the angle (2^-23 turn
    # of a circle for its fp32 form), relative to the row's largest element; far
    # positions: theta^(-2i/D) itself is a double here and there, pos * 2^-53
    err = 2.0 ** -19 + float(pos.max()) * 2.0 ** -50
    top = np.abs(yq).max(-1, keepdims=True)
    assert np.all(np.abs(f64(out) - yq) <= HALF[dtype] * np.abs(yq) + 2 * err * top
                  + (2.0 ** -25 if dtype == torch.float16 else 0))
    inplace = q.clone()
    if big > 1 << 24:
        assert int(st) == pkv.DEV_BAD_LEN
        return
    assert int(st) == 0
    gk, gv, gs = c.back()
    k, v, s = c.k.copy(), c.v.copy(), c.scales.copy()
    tab = np.concatenate([np.zeros((3, off), dtype=np.int32), table], 1)
    ref.append(k, v, s, yk, f64(vn), tab, pos, seq)
    assert np.array_equal(gv, v)
    assert np.array_equal(gs[..., 1], s[..., 1])
    moved = gs[..., 0] != s[..., 0]  # a largest element within err of a scale's limit
    assert moved.sum() <= 1
    for i in range(len(pos)):
        page, slot = tab[seq[i], pos[i] // P], pos[i] % P
        for h in range(Hkv):
            e = float(gs[page, h, slot // 16, 0]) - 127
            got = ref.VALUES[gk[page, h, slot]] * 2.0 ** e
            y = yk[i, h]
            lim = 2.0 ** -4 * np.abs(y) + 2.0 ** (e - 10) + 2 * err * np.abs(y).max()
            assert np.all(np.abs(got - y) <= lim)
    # rows of the touched pages that are no new rows: as the plain form leaves them
    mask = np.ones(gk.shape, dtype=bool)
    for i in range(len(pos)):
        mask[tab[seq[i], pos[i] // P], :, pos[i] % P] = False
    if not moved.any():
        assert np.array_equal(gk[mask], k[mask])
    pkv.kv8_append_rope(c.pool(), inplace, kn, vn, table_g, i32(pos), theta, inplace, i32(seq),
                        q_norm_weight=wq, k_norm_weight=wk, norm_eps=1e-5)
    assert torch.equal(inplace, out)
    again = c.back()
    assert all(np.array_equal(a, b) for a, b in zip(again, (gk, gv, gs))), "a second append"


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,count", [(128, [1777, 3090, 133]), (64, [4864]), (128, [4863, 1]),
                                     (64, [2000, 7777, 5, 18])])
def test_append_many_tokens(dtype, D, count):
    """More tokens than the device takes at once: the same bytes as a call a prompt."""
    Hq, Hkv, P = 64, 4, 32
    count = np.array(count)
    B = len(count)
    c = Cache(26, count, Hkv, D, P).gpu()
    one = Cache(26, count, Hkv, D, P).gpu()
    seq = np.repeat(np.arange(B), count)
    pos = np.concatenate([np.arange(n) for n in count])
    kn, vn = new_rows(c, len(pos), dtype)
    q = torch.randn(len(pos), Hq, D, device="cuda").to(dtype)
    wq = (1 + 0.2 * torch.randn(D)).to(dtype).cuda()
    out, two = torch.empty_like(q), torch.empty_like(q)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.kv8_append_rope(c.pool(), q, kn, vn, c.table_g, i32(pos), 10000.0, out, i32(seq),
                        dev_status=st, q_norm_weight=wq, k_norm_weight=wq)
    for b in range(B):
        x = slice(int(count[:b].sum()), int(count[:b + 1].sum()))
        for y in range(x.start, x.stop, 1600):  # pieces of whole blocks, each a small call
            z = slice(y, min(y + 1600, x.stop))
            pkv.kv8_append_rope(one.pool(), q[z], kn[z], vn[z], one.table_g, i32(pos[z]), 10000.0,
                                two[z], i32(seq[z]), dev_status=st, q_norm_weight=wq,
                                k_norm_weight=wq)
    assert int(st) == 0
    assert torch.equal(out, two)
    assert all(np.array_equal(a, b) for a, b in zip(c.back(), one.back()))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def check(c, q, out, scale, lens=None):
    """out [B][Q][Hq][D] against the plain form on the cache's numpy copy."""
    lens = c.lens if lens is None else lens
    qd = f64(q)
    want, mean, vmax = ref.attention(qd, c.k, c.v, c.scales, c.table, lens, scale)
    # scores: fp32 sums of D exact products (each partial sum rounds by 2^-24 of
    # the sum of magnitudes, at most D of them), and the exponent's own fp32 form
    top = np.abs(qd).sum(-1).max() * np.nanmax(np.abs(ref.VALUES[c.k])) * 2.0 ** (
        float(c.scales[..., 0].max()) - 127) * abs(scale) if c.lens.max() else 0.0
    score = min(1.0, top * 2.0 ** -24 * 6 + 2.0 ** -17)
    lim = ref.attention_bound(want, mean, vmax, lens, HALF[q.dtype], score)
    got = f64(out)
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > lim
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - want) - lim).max()),
                           np.argwhere(bad)[0])


def decode(c, q, scale, workers=0, stream=None):
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_kv8_workspace(q.shape[0], q.shape[1], c.Hkv, c.D, num_workers=workers)
    pkv.paged_decode_attention_kv8(q, c.k_g, c.v_g, c.s_g, c.table_g, c.lens_g, scale, out, ws,
                                   num_workers=workers)
    torch.cuda.synchronize()
    assert pkv.pkv_read_device_status(ws) == 0
    return out


SHAPES = [  # lens, Hq, Hkv, D, P
    ([1], 4, 2, 64, 16),
    ([37, 100], 4, 2, 64, 16),
    ([0, 1, 15, 16, 17, 0, 31, 32, 33, 250], 8, 2, 128, 16),
    ([500, 3, 77], 1, 1, 128, 32),
    ([300, 41], 7, 1, 128, 48),
    ([129, 64, 600], 12, 4, 64, 64),
    ([257, 90], 16, 1, 128, 256),
    ([333, 5, 0], 24, 1, 64, 32),
    ([210, 18], 32, 1, 128, 16),
    ([140, 333], 40, 1, 128, 16),   # a group of two units
    ([1000], 33, 1, 128, 16),       # a group cut into threes of eleven
    ([900, 1200, 40], 28, 4, 128, 32),
    ([50, 2000], 9, 3, 64, 128),
    ([2500, 2490], 512, 16, 64, 16),  # few units, many rows
    ([700], 64, 1, 128, 16),          # a group that fills half a tensor-core tile
    ([90, 1500, 0, 17], 96, 1, 64, 32),
    ([640, 33], 260, 2, 128, 48),     # 130 rows a KV head: two tiles
    ([1200] * 16 + [1111], 32, 1, 128, 16),  # parts merged in their CTA, a warp a row after
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("workers", [0, 1, 7])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P", SHAPES)
def test_decode(dtype, workers, lens, Hq, Hkv, D, P):
    c = Cache(7, lens, Hkv, D, P).poison().gpu()
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    out = decode(c, q, D ** -0.5, workers)
    check(c, q[:, None], out[:, None], D ** -0.5)
    assert (out[c.lens_g == 0] == 0).all()


@pytest.mark.parametrize("Hq", [6, 20, 70])
@pytest.mark.parametrize("dtype", DT)
def test_decode_scales_apart(dtype, Hq):
    """V scales from one end of their range to the other in one sequence: fp16
    outputs need the values small, so the large ones go with small weights."""
    c = Cache(8, [400, 200], 1, 128, 16)
    c.scales[..., 1] = c.rng.integers(127 - 60, 127 + 41 if dtype == torch.bfloat16 else 127 + 4,
                                      c.scales[..., 1].shape)
    c.gpu()
    q = torch.randn(2, Hq, 128, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    check(c, q[:, None], decode(c, q, 0.1)[:, None], 0.1)


@pytest.mark.parametrize("Hq", [3, 70])
def test_decode_negative_and_zero_scale(Hq):
    c = Cache(23, [300, 33], 1, 128, 16).gpu()
    for dtype in DT:
        q = torch.randn(2, Hq, 128, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
        for scale in (-0.09, 0.0):
            check(c, q[:, None], decode(c, q, scale)[:, None], scale)


def test_decode_large_batches():
    """More sequences than a CTA plans for itself (the plan kernel's path), with
    empty ones, padded lengths and a bad length among them."""
    B = 700
    lens = np.random.default_rng(5).integers(0, 70, B)
    lens[::9] = 0
    c = Cache(24, lens, 2, 64, 16).poison().gpu()
    for Hq in (6, 140):
        q = torch.randn(B, Hq, 64, generator=torch.Generator().manual_seed(4)).half().cuda()
        out = decode(c, q, 0.125)
        sel = np.r_[0:40, B - 20:B]
        sub = Cache.__new__(Cache)
        sub.__dict__.update(c.__dict__)
        sub.table, sub.lens = c.table[sel], c.lens[sel]
        check(sub, q[sel][:, None], out[sel][:, None], 0.125)
        bad = c.lens_g.clone()
        bad[3] = -5
        ws = pkv.alloc_kv8_workspace(B, Hq, 2, 64)
        two = torch.empty_like(out)
        pkv.paged_decode_attention_kv8(q, c.k_g, c.v_g, c.s_g, c.table_g, bad, 0.125, two, ws)
        assert pkv.pkv_read_device_status(ws) == pkv.DEV_BAD_LEN
        assert (two[3] == 0).all()


@pytest.mark.parametrize("B", [511, 512, 513])
@pytest.mark.parametrize("Hq", [4, 140])
def test_decode_batches_around_the_plan(B, Hq):
    """The largest batches whose ranges every CTA works out, the smallest beyond."""
    lens = np.random.default_rng(B).integers(0, 50, B)
    lens[-1] = 41
    c = Cache(25, lens, 2, 64, 16).poison().gpu()
    q = torch.randn(B, Hq, 64, generator=torch.Generator().manual_seed(4)).half().cuda()
    out = decode(c, q, 0.125)
    sel = np.r_[0:20, B - 20:B]
    sub = Cache.__new__(Cache)
    sub.__dict__.update(c.__dict__)
    sub.table, sub.lens = c.table[sel], c.lens[sel]
    check(sub, q[sel][:, None], out[sel][:, None], 0.125)
    assert (out[c.lens_g == 0] == 0).all()


@pytest.mark.parametrize("long", [500, 1100, 9000])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_one_long_among_many(long, D):
    """One sequence of many segments (tens to hundreds) where most have one."""
    lens = np.array([3] * 100 + [long] + [3] * 155)
    c = Cache(27, lens, 2, D, 16).poison().gpu()
    q = torch.randn(256, 8, D, generator=torch.Generator().manual_seed(4)).half().cuda()
    check(c, q[:, None], decode(c, q, 0.1)[:, None], 0.1)


def test_decode_queries_of_any_size():
    """bf16 queries far outside fp16's range, zero rows and mixed sizes in a row."""
    c = Cache(9, [100, 300, 64], 2, 128, 16).gpu()
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(5))
    q *= torch.exp2(torch.linspace(-30, 30, 8)).view(1, 8, 1)
    q[:, 3] = 0
    q[:, 5, ::3] *= 2.0 ** -20
    q = q.bfloat16().cuda()
    for h in range(8):
        scale = float(2.0 ** -(h * 60 / 7 - 30)) * 0.05
        out = decode(c, q, scale)
        one = Cache.__new__(Cache)
        one.__dict__.update(c.__dict__)
        want, mean, vmax = ref.attention(f64(q)[:, None], c.k, c.v, c.scales, c.table, c.lens, scale)
        lim = ref.attention_bound(want, mean, vmax, c.lens, 2.0 ** -8, 2.0 ** -12)
        sel = np.s_[:, 0, h]
        assert np.all(np.abs(f64(out)[:, h] - want[sel]) <= lim[sel]), h


def test_decode_nan_where_seen_only():
    """A NaN in an attended value or key reaches its own head's rows, no other."""
    c = Cache(10, [40, 70], 2, 128, 16).poison()
    c.v[c.table[0, 1], 1, 3, 17] = 0x7F      # sequence 0, head 1, token 19
    c.k[c.table[1, 4], 0, 5, 100] = 0xFF     # sequence 1, head 0, token 69
    c.gpu()
    q = torch.randn(2, 8, 128).bfloat16().cuda()
    out = decode(c, q, 0.09)
    nan = out.isnan()
    want = torch.zeros_like(nan)
    want[0, 4:, 17] = True
    want[1, :4] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("workers", [0, 3])
@pytest.mark.parametrize("Q,lens,Hq,Hkv,D,P", [
    (1, [40, 0, 7], 8, 2, 128, 16),
    (2, [1, 2, 3, 50, 0], 4, 2, 64, 16),
    (5, [5, 33, 300], 8, 2, 128, 32),
    (8, [200, 9, 3], 4, 1, 128, 16),       # 32 rows a unit
    (7, [64, 130], 7, 1, 64, 48),
    (16, [16, 400], 6, 3, 128, 16),
    (33, [33, 20, 210], 4, 2, 128, 64),    # two query tiles
    (64, [64, 500, 10], 8, 2, 128, 16),
    (64, [128, 70], 3, 1, 64, 256),
    (3, [90, 1000], 32, 1, 128, 16),
    (40, [41, 700, 2, 0, 129], 4, 2, 128, 16),   # 80 rows a KV head
    (64, [2000, 1], 5, 1, 64, 64),               # 320 rows: three tiles
    (17, [400, 18], 24, 3, 128, 48),             # 136 rows
    (8, [1500, 900, 1211], 32, 8, 128, 16),      # parts merged in their CTA
    (3, [1500, 700, 9, 1211, 900], 48, 8, 64, 32),
    (12, [800, 90], 8, 2, 128, 16),              # the most rows of the warp kernel
    (7, [800, 90], 14, 2, 64, 16),               # the fewest of the tensor-core tile
])
def test_multi(dtype, workers, Q, lens, Hq, Hkv, D, P):
    c = Cache(11, lens, Hkv, D, P).poison().gpu()
    q = torch.randn(len(lens), Q, Hq, D, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_kv8_workspace(len(lens), Hq, Hkv, D, n_queries=Q, num_workers=workers)
    pkv.paged_decode_attention_multi_kv8(q, c.k_g, c.v_g, c.s_g, c.table_g, c.lens_g, D ** -0.5,
                                         out, ws, num_workers=workers)
    assert pkv.pkv_read_device_status(ws) == 0
    check(c, q, out, D ** -0.5)
    for b, n in enumerate(lens):
        assert (out[b, :max(0, Q - n)] == 0).all(), "queries before the first token"
    if Q == 1:
        assert torch.equal(out[:, 0], decode(c, q[:, 0].contiguous(), D ** -0.5, workers))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,n", [(4, 30), (4, 200), (8, 30), (8, 150), (8, 1000)])
def test_multi_nan_in_a_later_token(Hq, n, D):
    """A NaN in the value of one of the queries' own tokens reaches only the
    queries from there on, also through weights that vanish; one far before
    them reaches all (48 rows: the warp kernel; 96: the tensor-core tile)."""
    Q = 12  # queries stand at the last 12 tokens
    at = n - 10
    c = Cache(12, [n, n], 1, D, 16).poison()
    c.v[c.table[0, at // 16], 0, at % 16, 5] = 0x7F
    c.v[c.table[1, 0], 0, 7, D - 1] = 0xFF
    c.gpu()
    q = torch.randn(2, Q, Hq, D).half().cuda()
    for workers in (0, 1):
        out = torch.empty_like(q)
        ws = pkv.alloc_kv8_workspace(2, Hq, 1, D, n_queries=Q, num_workers=workers)
        pkv.paged_decode_attention_multi_kv8(q, c.k_g, c.v_g, c.s_g, c.table_g, c.lens_g, 0.09,
                                             out, ws, num_workers=workers)
        want = torch.zeros_like(out, dtype=torch.bool)
        want[0, 2:, :, 5] = True
        want[1, :, :, D - 1] = True
        assert torch.equal(out.isnan(), want)


@pytest.mark.parametrize("Hq", [8, 140])
def test_attention_bad_inputs(Hq):
    """Bad page ids and lengths are flagged; the other sequences are unharmed."""
    c = Cache(13, [100, 90, 60], 2, 128, 16).gpu()
    q = torch.randn(3, Hq, 128).bfloat16().cuda()
    good = decode(c, q, 0.09)
    c.table_g[1, 2] = c.NP + 5
    lens = c.lens_g.clone()
    lens[2] = 1000  # beyond the table row: clamped to it, whose last entries are -1
    out = torch.empty_like(q)
    ws = pkv.alloc_kv8_workspace(3, Hq, 2, 128)
    pkv.paged_decode_attention_kv8(q, c.k_g, c.v_g, c.s_g, c.table_g, lens, 0.09, out, ws)
    assert pkv.pkv_read_device_status(ws) == pkv.DEV_BAD_PAGE | pkv.DEV_BAD_LEN
    assert (out[0] - good[0]).abs().max() < 0.02 * good[0].abs().max()
    assert out.isfinite().all()


@pytest.mark.parametrize("B", [1, 300, 600])
@pytest.mark.parametrize("group", [1, 64])
def test_more_positions_than_32_bits(B, group):
    """A batch whose chunks over all heads do not fit 32 bits is refused on the
    device: flagged, and zeros."""
    Hkv, D, P, n = 4096 // group, 64, 16, 16 * (600000 if B == 1 else 2000) * group
    k = torch.zeros((2, Hkv, P, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((2, Hkv, 1, 2), 127, dtype=torch.uint8, device="cuda").view(
        torch.float8_e8m0fnu)
    table = torch.zeros((B, n // P), dtype=torch.int32, device="cuda")
    q = torch.randn(B, Hkv * group, D).half().cuda()
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_kv8_workspace(B, Hkv * group, Hkv, D)
    pkv.paged_decode_attention_kv8(q, k, k, s, table, i32([n] * B), 0.1, out, ws)
    assert pkv.pkv_read_device_status(ws) == pkv.DEV_BAD_LEN
    assert (out == 0).all()


@pytest.mark.parametrize("Hq", [8, 140])
def test_page_ids_and_reruns_do_not_matter(Hq):
    c = Cache(14, [700, 30, 260], 2, 128, 32).gpu()
    q = torch.randn(3, Hq, 128).half().cuda()
    a, b = decode(c, q, 0.09), decode(c, q, 0.09)
    assert torch.equal(a, b)
    perm = torch.from_numpy(c.rng.permutation(c.NP)).cuda()
    inv = torch.argsort(perm)
    move = lambda t: t.view(torch.uint8)[perm].contiguous().view(t.dtype)  # noqa: E731
    d = Cache.__new__(Cache)
    d.__dict__.update(c.__dict__)
    d.k_g, d.v_g, d.s_g = move(c.k_g), move(c.v_g), move(c.s_g)
    d.table_g = torch.where(c.table_g >= 0, inv[c.table_g.clamp(min=0).long()].int(), c.table_g)
    assert torch.equal(decode(d, q, 0.09), a)


# ---------------------------------------------------------------------------
# the step, and the operators together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("theta,norm", [(0.0, False), (10000.0, False), (500000.0, True)])
@pytest.mark.parametrize("Hq,Hkv,D,P", [(8, 2, 128, 16), (28, 4, 128, 32), (4, 4, 64, 48)])
def test_step_equals_append_then_attention(dtype, theta, norm, Hq, Hkv, D, P):
    lens = [33, 1, 0, 400, 16, 17, 900]
    a, b = (Cache(15, lens, Hkv, D, P).gpu() for _ in range(2))
    pos = i32(np.array(lens) - 1)
    pos[4] = -1  # attends, but appends nothing
    kn, vn = new_rows(a, len(lens), dtype)
    q = torch.randn(len(lens), Hq, D).to(dtype).cuda()
    w = [(1 + 0.1 * torch.randn(D)).to(dtype).cuda() if norm else None for _ in range(2)]
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_kv8_workspace(len(lens), Hq, Hkv, D)
    keep = q.clone()
    pkv.paged_decode_step_kv8(kn, vn, pos, q, a.k_g, a.v_g, a.s_g, a.table_g, a.lens_g, D ** -0.5,
                              out, ws, rope_theta=theta, q_norm_weight=w[0], k_norm_weight=w[1])
    assert pkv.pkv_read_device_status(ws) == 0 and torch.equal(q, keep)
    if theta:
        q2 = torch.empty_like(q)
        pkv.kv8_append_rope(b.pool(), q, kn, vn, b.table_g, pos, theta, q2, q_norm_weight=w[0],
                            k_norm_weight=w[1])
    else:
        q2 = q
        pkv.kv8_append(b.pool(), kn, vn, b.table_g, pos)
    for x, y in zip(a.back(), b.back()):
        assert np.array_equal(x, y)
    want = decode(b, q2, D ** -0.5)
    assert torch.equal(out, want)
    b.k, b.v, b.scales = b.back()
    check(b, q2[:, None], out[:, None], D ** -0.5)


def test_step_reports_append_errors():
    c = Cache(16, [20, 40, 30], 2, 64, 16).gpu()
    kn, vn = new_rows(c, 3, torch.float16)
    q = torch.randn(3, 4, 64).half().cuda()
    out = torch.empty_like(q)
    ws = pkv.alloc_kv8_workspace(3, 4, 2, 64)
    call = lambda pos: pkv.paged_decode_step_kv8(  # noqa: E731
        kn, vn, i32(pos), q, c.k_g, c.v_g, c.s_g, c.table_g, c.lens_g, 0.125, out, ws)
    call([19, 5000, 29])
    assert pkv.pkv_read_device_status(ws) == pkv.DEV_BAD_LEN
    call([19, 39, 29])
    assert pkv.pkv_read_device_status(ws) == 0


def test_requests_from_prompt_to_decode():
    """Prompts of several requests appended in pieces of up to 64 tokens, each
    piece attended by its own queries, then decode steps: against the plain
    forms run over the same tokens from the start."""
    D, Hq, Hkv, P, theta = 64, 4, 2, 16, 10000.0
    dtype = torch.bfloat16
    prompts = np.array([150, 64, 7])
    steps = 20
    c = Cache(17, prompts, Hkv, D, P, cap=prompts + steps)
    c.k[:], c.v[:], c.scales[:] = 0x7F, 0x7F, 255  # nothing there yet
    c.gpu()
    pool = c.pool()
    gen = torch.Generator().manual_seed(8)
    mk = lambda *s: torch.randn(*s, generator=gen).to(dtype).cuda()  # noqa: E731
    done = np.zeros(3, dtype=np.int64)
    k, v, s = c.k.copy(), c.v.copy(), c.scales.copy()

    def compare(q_rot, out, lens):
        c.k, c.v, c.scales = c.back()
        c.lens = np.asarray(lens, dtype=np.int32)
        check(c, q_rot, out, D ** -0.5)

    while (done < prompts).any():
        Q = 64
        n = np.minimum(prompts - done, Q)
        seq = np.repeat(np.arange(3), n)
        pos = np.concatenate([np.arange(a, a + m) for a, m in zip(done, n)])
        q, kn, vn = mk(len(pos), Hq, D), mk(len(pos), Hkv, D), mk(len(pos), Hkv, D)
        q_rot = torch.empty_like(q)
        pkv.kv8_append_rope(pool, q, kn, vn, c.table_g, i32(pos), theta, q_rot, i32(seq))
        ref.append(k, v, s, ref.norm_rope(f64(kn), None, pos, theta, 0.0), f64(vn), c.table, pos,
                   seq)
        done += n
        # queries end at each request's last token: pad in front
        qs = torch.zeros(3, Q, Hq, D, dtype=dtype, device="cuda")
        for b in range(3):
            if n[b]:
                qs[b, Q - n[b]:] = q_rot[i32(seq) == b]
        out = torch.empty_like(qs)
        ws = pkv.alloc_kv8_workspace(3, Hq, Hkv, D, n_queries=Q)
        pkv.paged_decode_attention_multi_kv8(qs, c.k_g, c.v_g, c.s_g, c.table_g, i32(done),
                                             D ** -0.5, out, ws)
        compare(qs, out, done)
    ws = pkv.alloc_kv8_workspace(3, Hq, Hkv, D)
    out = torch.empty(3, Hq, D, dtype=dtype, device="cuda")
    for _ in range(steps):
        q, kn, vn = mk(3, Hq, D), mk(3, Hkv, D), mk(3, Hkv, D)
        pkv.paged_decode_step_kv8(kn, vn, i32(done), q, c.k_g, c.v_g, c.s_g, c.table_g,
                                  i32(done + 1), D ** -0.5, out, ws, rope_theta=theta)
        ref.append(k, v, s, ref.norm_rope(f64(kn), None, done, theta, 0.0), f64(vn), c.table,
                   done, np.arange(3))
        y = ref.norm_rope(f64(q), None, done, theta, 0.0)
        done = done + 1
    assert pkv.pkv_read_device_status(ws) == 0
    gk, gv, gs = c.back()
    assert np.array_equal(gv, v) and np.array_equal(gs[..., 1], s[..., 1])
    # keys: at most one e4m3 step apart where the exact rotation lies at a border
    assert (gk != k).mean() < 1e-3
    # the queries were rotated in the step: bf16 of the exact rotation, give or take a step
    compare(torch.from_numpy(y).to(dtype).cuda()[:, None], out[:, None], done)


# ---------------------------------------------------------------------------
# streams, graphs, workspaces
# ---------------------------------------------------------------------------
def test_graph_replay_with_new_lengths_and_two_graphs():
    """A captured step follows the lengths, positions and rows in its buffers;
    two graphs with a workspace each, replayed on two streams at once."""
    lens = np.array([200, 64, 33, 1])
    graphs = []
    for seed in (18, 19):
        c = Cache(seed, lens, 2, 128, 16, cap=lens + 20).gpu()
        kn, vn = new_rows(c, 4, torch.float16)
        q = torch.randn(4, 8, 128).half().cuda()
        out = torch.empty_like(q)
        ws = pkv.alloc_kv8_workspace(4, 8, 2, 128)
        pos, ln = i32(lens - 1), i32(lens)
        args = (kn, vn, pos, q, c.k_g, c.v_g, c.s_g, c.table_g, ln, 0.09, out, ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            pkv.paged_decode_step_kv8(*args, rope_theta=1e4)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_decode_step_kv8(*args, rope_theta=1e4)
        graphs.append((c, g, args, side))
    for step in range(3):
        for c, g, args, side in graphs:
            kn, vn = new_rows(c, 4, torch.float16)
            args[0].copy_(kn)
            args[1].copy_(vn)
            args[2].copy_(i32(lens + step))
            args[8].copy_(i32(lens + step + 1))
        torch.cuda.synchronize()
        before = [[t.clone() for t in (c.k_g, c.v_g, c.s_g)] for c, *_ in graphs]
        for c, g, args, side in graphs:
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for (c, g, args, side), (k, v, s) in zip(graphs, before):
            out = torch.empty_like(args[10])
            ws = pkv.alloc_kv8_workspace(4, 8, 2, 128)
            pkv.paged_decode_step_kv8(*args[:4], k, v, s, *args[7:10], out, ws, rope_theta=1e4)
            assert torch.equal(out, args[10])
            for x, y in ((k, c.k_g), (v, c.v_g), (s, c.s_g)):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_given_stream_is_the_one_used():
    c = Cache(20, [3000, 2000], 2, 128, 16).gpu()
    q = torch.randn(2, 8, 128).bfloat16().cuda()
    want = decode(c, q, 0.09)
    side = torch.cuda.Stream()
    out = torch.zeros_like(q)
    ws = pkv.alloc_kv8_workspace(2, 8, 2, 128)
    late = torch.empty_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)  # the call must come after this
    pkv.paged_decode_attention_kv8(late, c.k_g, c.v_g, c.s_g, c.table_g, c.lens_g, 0.09, out, ws,
                                   stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_binding_refuses():
    c = Cache(21, [20, 30], 2, 64, 16).gpu()
    q = torch.randn(2, 4, 64).half().cuda()
    out, ws = torch.empty_like(q), pkv.alloc_kv8_workspace(2, 4, 2, 64)
    good = dict(q=q, k_pool=c.k_g, v_pool=c.v_g, scales=c.s_g, page_table=c.table_g,
                context_lens=c.lens_g, scale=0.1, out=out, workspace=ws)
    pkv.paged_decode_attention_kv8(**good)
    for name, bad in [("q", q.float()), ("q", q[:, ::2]), ("q", q[:1]), ("out", out.bfloat16()),
                      ("k_pool", c.k_g.view(torch.uint8)), ("scales", c.s_g[:, :1]),
                      ("scales", c.s_g.view(torch.uint8).int()), ("context_lens", c.lens_g.long()),
                      ("context_lens", c.lens_g[:1]), ("page_table", c.table_g.cpu()),
                      ("workspace", ws.cpu())]:
        with pytest.raises(ValueError):
            pkv.paged_decode_attention_kv8(**dict(good, **{name: bad}))
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_decode_attention_kv8(**dict(good, workspace=ws[:256]))
    assert e.value.name == "PKV_ERR_WORKSPACE"
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_decode_attention_kv8(**dict(good, out=q))
    assert e.value.name == "PKV_ERR_ALIAS"
    pool = c.pool()
    kn, vn = new_rows(c, 2, torch.float16)
    with pytest.raises(ValueError):
        pkv.kv8_append(pool, kn.float(), vn.float(), c.table_g, i32([0, 0]))
    with pytest.raises(ValueError):
        pkv.kv8_append(pool, kn, vn, c.table_g[:1].contiguous(), i32([0, 0]))
    with pytest.raises(ValueError):
        pkv.kv8_append(pool, kn, vn, c.table_g, i32([0, 0]), i32([0]))
    with pytest.raises(ValueError):
        pkv.kv_append(pool, kn, vn, c.table_g, i32([0, 0]))
    own = pkv.kv8_pool_create(4, 16, 2, 64)  # memory of its own
    assert own.k_ptr() and own.v_ptr() and own.scales_ptr()
    own.destroy()


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes a side, its last pages in use."""
    D, P, Hkv = 128, 256, 8
    NP = (1 << 32) // (P * Hkv * D) + 40
    k = torch.empty((NP, Hkv, P, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.empty((NP, Hkv, P, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((NP, Hkv, P // 16, 2), 127, dtype=torch.uint8, device="cuda").view(
        torch.float8_e8m0fnu)
    small = Cache(22, [500, 300], Hkv, D, P).gpu()
    n = small.NP
    for big, t in ((k, small.k_g), (v, small.v_g), (s, small.s_g)):
        big.view(torch.uint8)[NP - n:] = t.view(torch.uint8)
    table = torch.where(small.table_g >= 0, small.table_g + (NP - n), small.table_g)
    kn, vn = new_rows(small, 2, torch.bfloat16)
    q = torch.randn(2, 16, D).bfloat16().cuda()
    outs = []
    for kk, vv, ss, tt in ((k, v, s, table), (small.k_g, small.v_g, small.s_g, small.table_g)):
        out = torch.empty_like(q)
        ws = pkv.alloc_kv8_workspace(2, 16, Hkv, D)
        pkv.paged_decode_step_kv8(kn, vn, i32([499, 299]), q, kk, vv, ss, tt, small.lens_g, 0.09,
                                  out, ws, rope_theta=1e4)
        assert pkv.pkv_read_device_status(ws) == 0
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(k.view(torch.uint8)[NP - n:], small.k_g.view(torch.uint8))

"""Attention over an 8-bit cache whose V scales lie far apart inside a sequence: every
output within a bound made of each token's own value and weight (kv8_bound)."""
import numpy as np
import pytest
import torch

import kv8_bound as kb
import paged_kv_decode_16_gb300 as pkv
from test_gpu_kv8 import Cache

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def run(c, q, scale, workers=0):
    """q [B][Q][Hq][D] -> the kernels' output."""
    B, Q, Hq, D = q.shape
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_kv8_workspace(B, Hq, c.Hkv, D, n_queries=Q, num_workers=workers)
    pkv.paged_decode_attention_multi_kv8(q, c.k_g, c.v_g, c.s_g, c.table_g, c.lens_g, scale, out,
                                         ws, num_workers=workers)
    assert pkv.pkv_read_device_status(ws) == 0
    return out


def outliers(seed, lens, D, at, size, weight, unit=1.0, H=1, P=16):
    """A cache of normal values, times `unit`, but for one element of one token (at) of every
    sequence, which is `size`; that token's weight is about e^weight of the others'.
    Queries have element 0 equal to 4 in every row."""
    c = Cache(seed, lens, H, D, P)
    k, v = [], []
    for n in lens:
        x = c.rng.standard_normal((2, n, H, D))
        x[1] *= unit
        x[0, :, :, 0] = 0.0
        if at < n:
            x[0, at, :, 0] = weight / 4.0 * D ** 0.5
            x[1, at, :, 7] = size
        k.append(x[0])
        v.append(x[1])
    return kb.fill(c, k, v).poison().gpu()


def queries(B, Q, Hq, D, dtype, seed=3):
    q = torch.randn(B, Q, Hq, D, generator=torch.Generator().manual_seed(seed)).double()
    q[..., 0] = 4.0
    return q.to(dtype).cuda()


@pytest.mark.parametrize("workers", [0, 1, 3])
@pytest.mark.parametrize("Hq", [6, 12, 20, 70])  # tiles of 8, 16, 24 rows; the tensor-core tile
@pytest.mark.parametrize("k", [12, 16, 20, 24, 28, 40])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (FP, 128), (FP, 64)])
def test_outlier_of_negligible_weight(dtype, D, k, Hq, workers):
    lens = [512, 700, 90]
    for at in (37, 300):
        c = outliers(30, lens, D, at, 2.0 ** k, -50.0)
        q = queries(3, 1, Hq, D, dtype)
        kb.check(c, q, run(c, q, D ** -0.5, workers), D ** -0.5)


@pytest.mark.parametrize("workers", [0, 1])
@pytest.mark.parametrize("Hq", [6, 12, 20, 70])
@pytest.mark.parametrize("dtype,k", [(BF, 12), (BF, 20), (BF, 28), (BF, 40), (FP, 12), (FP, 20),
                                     (FP, 24)])
def test_outlier_of_ordinary_weight(dtype, k, Hq, workers):
    D = 128
    # fp16: the outlier's own output must fit, so the others are small
    unit = 1.0 if dtype == BF else 2.0 ** min(0, 15 - k)
    c = outliers(31, [600, 900], D, 100, 2.0 ** k * unit, 0.0, unit)
    q = queries(2, 1, Hq, D, dtype)
    kb.check(c, q, run(c, q, D ** -0.5, workers), D ** -0.5)


@pytest.mark.parametrize("workers", [0, 1])
@pytest.mark.parametrize("Hq", [6, 70])
@pytest.mark.parametrize("k", [16, 28])
def test_outlier_in_a_long_sequence(k, Hq, workers):
    c = outliers(32, [4096], 128, 1500, 2.0 ** k, -50.0)
    q = queries(1, 1, Hq, 128, BF)
    kb.check(c, q, run(c, q, 128 ** -0.5, workers), 128 ** -0.5)


@pytest.mark.parametrize("workers", [0, 1])
@pytest.mark.parametrize("Hq", [6, 12, 20, 70])
@pytest.mark.parametrize("dtype,spread", [(BF, 20), (BF, 40), (FP, 8)])
def test_every_block_a_scale_of_its_own(dtype, spread, Hq, workers):
    """Values of 2^-spread to 2^spread, a size a block, with weights that make the blocks
    count alike in the output."""
    D, n = 64, 500
    c = Cache(33, [n, 77], 2, D, 32)
    k, v = [], []
    for n in c.lens:
        x = c.rng.standard_normal((2, n, 2, D))
        e = np.repeat(c.rng.integers(-spread, spread + 1, (-(-n // 16), 2)), 16, axis=0)[:n]
        x[1] *= 2.0 ** e[..., None]
        x[0, :, :, 0] = -e * np.log(2.0) / 4.0 * D ** 0.5
        k.append(x[0])
        v.append(x[1])
    kb.fill(c, k, v).poison().gpu()
    q = queries(2, 1, 2 * Hq, D, dtype)
    kb.check(c, q, run(c, q, D ** -0.5, workers), D ** -0.5)


@pytest.mark.parametrize("workers", [0, 1])
@pytest.mark.parametrize("Q,Hq", [(5, 4), (12, 4), (12, 8), (40, 5)])
@pytest.mark.parametrize("at", [0, 130, 195])  # far before the queries, and among them
def test_several_queries(at, Q, Hq, workers):
    c = outliers(34, [200, 340], 128, at, 2.0 ** 24, -50.0)
    q = queries(2, Q, Hq, 128, FP)
    kb.check(c, q, run(c, q, 128 ** -0.5, workers), 128 ** -0.5)


@pytest.mark.parametrize("workers", [0, 1])
@pytest.mark.parametrize("Hq", [4, 8])
def test_several_queries_and_a_nan(Hq, workers):
    """A NaN in a later token's value beside an outlier: it reaches the queries that see
    it, in its own channel; everything else is within the bound."""
    D, Q, n = 128, 12, 200
    c = outliers(35, [n, 170], D, 40, 2.0 ** 24, -50.0)
    at = n - 5
    c.v[c.table[0, at // 16], 0, at % 16, 9] = 0x7F
    c.gpu()
    q = queries(2, Q, Hq, D, FP)
    out = run(c, q, D ** -0.5, workers)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[0, Q - 5:, :, 9] = True
    assert torch.equal(out.isnan(), nan)
    c.v[c.table[0, at // 16], 0, at % 16, 9] = 0
    out[nan] = 0.0
    want, lim = kb.attention(q.double().cpu().numpy(), c.k, c.v, c.scales, c.table, c.lens,
                             D ** -0.5, "float16")
    keep = ~nan.cpu().numpy()
    assert (np.abs(out.double().cpu().numpy() - want) <= lim)[keep].all()


@pytest.mark.parametrize("Hq", [6, 70])
def test_blocks_of_zeros_and_bad_pages(Hq):
    """Blocks that hold zeros (the smallest scale), and pages that are skipped, beside
    ordinary ones."""
    D = 128
    c = Cache(36, [300, 200], 1, D, 16)
    k, v = [], []
    for n in c.lens:
        x = c.rng.standard_normal((2, n, 1, D))
        x[0, :, :, 0] = 0.0
        x[1, 32:96] = 0.0
        x[1, 5, :, 3] = 2.0 ** 22
        x[0, 5, :, 0] = -50.0 / 4.0 * D ** 0.5
        k.append(x[0])
        v.append(x[1])
    kb.fill(c, k, v).gpu()
    q = queries(2, 1, Hq, D, BF)
    kb.check(c, q, run(c, q, D ** -0.5), D ** -0.5)
    # page 9 of sequence 1 is bad: as if its tokens were not there
    c.table_g[1, 9] = c.NP
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_kv8_workspace(2, Hq, 1, D)
    pkv.paged_decode_attention_multi_kv8(q, c.k_g, c.v_g, c.s_g, c.table_g, c.lens_g, D ** -0.5,
                                         out, ws)
    assert pkv.pkv_read_device_status(ws) == pkv.DEV_BAD_PAGE
    short = Cache.__new__(Cache)
    short.__dict__.update(c.__dict__)
    short.table, short.lens = c.table.copy(), c.lens.copy()
    short.table[1, 9:-1] = c.table[1, 10:]
    short.lens[1] -= 16
    kb.check(short, q, out, D ** -0.5)


@pytest.mark.parametrize("workers", [0, 1])
@pytest.mark.parametrize("Hq", [6, 20, 70])
@pytest.mark.parametrize("weight", [-100.0, -20.0, 0.0])
def test_scales_from_one_end_to_the_other(weight, Hq, workers):
    """Values of 2^-52 with one of 2^47 every 40 tokens: of weights that leave nothing of
    it, that share the output, and that make up its channel."""
    D = 128
    c = Cache(37, [330, 170], 1, D, 16)
    k, v = [], []
    for n in c.lens:
        x = c.rng.standard_normal((2, n, 1, D))
        x[0, :, :, 0] = 0.0
        x[0, 7::40, :, 0] = weight / 4.0 * D ** 0.5
        x[1] *= 2.0 ** -52
        x[1, 7::40, :, 7] = 2.0 ** 47
        k.append(x[0])
        v.append(x[1])
    kb.fill(c, k, v).poison().gpu()
    q = queries(2, 1, Hq, D, BF)
    kb.check(c, q, run(c, q, D ** -0.5, workers), D ** -0.5)

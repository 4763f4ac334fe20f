"""The weights of the attention over selected pages: both 16-bit pieces of them, their range,
and values that are not finite."""
import math
import random

import pytest
import torch

import selected_bound as sb
import selected_ref as ref
from test_gpu_selected import (BF16, DEV, F16, i32, page_table, rand, run_attend, some_lists,
                               status_word)

pytestmark = pytest.mark.gpu


def check(q, k, v, table, lens, lists, scale):
    q, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    st = status_word()
    got = run_attend(q, k, v, i32(table), i32(lens), i32(lists), scale, st)
    ref.close(got, *sb.attend(q, k, v, table, lens, lists, scale))
    assert st.item() == 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("seed", range(5))
def test_attend_outputs_that_cancel(dtype, seed):
    check(*sb.cancelling(dtype, seed))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("drop", [12, 20, 22, 25, 26, 28, 32])
def test_attend_long_tail_of_small_weights(dtype, drop):
    check(*sb.tail(dtype, drop))


@pytest.mark.parametrize("hq,hkv,d,page,dtype,keep,lens", [
    (4, 2, 64, 16, F16, 8, [37, 100]),
    (32, 8, 128, 16, BF16, 40, [0, 1, 15, 16, 17, 3000, 640]),
    (28, 4, 128, 32, F16, 20, [161, 5000, 31]),
    (20, 1, 64, 48, F16, 7, [9000, 49, 200]),
    (34, 2, 64, 16, BF16, 33, [900, 100]),
    (12, 4, 128, 16, F16, 12, [17 * i for i in range(60)]),
])
def test_attend_within_the_bound_of_two_pieces(hq, hkv, d, page, dtype, keep, lens):
    gen = torch.Generator(device=DEV).manual_seed(hq)
    rng = random.Random(hq)
    NP = sum(-(-n // page) for n in lens) + 2
    cols = max(-(-n // page) for n in lens) + 1
    table = page_table(rng, lens, page, NP, cols)
    k, v = (rand(gen, NP, hkv, page, d, dtype=dtype) for _ in range(2))
    check(rand(gen, len(lens), hq, d, dtype=dtype), k, v, table, lens,
          some_lists(rng, lens, hkv, page, keep), d ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,keep", [(40, 3), (1600, 100)])
def test_attend_infinite_values(dtype, n, keep):
    """An infinity in V under a weight that is not 0 makes its element infinite, two of
    unequal signs NaN, whatever the weight: 1, of few bits, or of many."""
    gen = torch.Generator(device=DEV).manual_seed(n)
    pages = -(-n // 16)
    k, v = (rand(gen, pages, 1, 16, 64, dtype=dtype) for _ in range(2))
    q = torch.zeros(1, 4, 64, dtype=dtype, device=DEV)
    q[0, :, 0] = torch.tensor([1.0, 2.0, 0.0, -1.0])
    k[..., 0] = torch.randint(-3, 4, (pages, 1, 16), generator=gen, device=DEV).to(dtype)
    k[..., 0][1, 0, 3] = 0.7
    k[..., 0][0, 0, 3] = 4.0                      # the largest score: a weight of 1
    for t, (d, x) in enumerate([(1, math.inf), (2, -math.inf), (3, math.inf), (3, -math.inf)]):
        v[0, 0, 3 + t, d] = x
    v[1, 0, 3, 4] = math.inf                      # a weight of many bits
    v[2, 0, 1, 5] = -math.inf
    table, lists = [list(range(pages))], [[list(range(pages)) + [-1] * (keep - pages)]]
    got = run_attend(q, k, v, i32(table), i32([n]), i32(lists), math.log(2.0))
    x = got[0].float()
    assert (x[:, 1] == math.inf).all() and (x[:, 2] == -math.inf).all() and x[:, 3].isnan().all()
    assert (x[:, 4] == math.inf).all() and (x[:, 5] == -math.inf).all()
    fine = [0] + list(range(6, 64))
    v[..., 1:6] = 0.0
    want, bound = sb.attend(q, k, v, table, [n], lists, math.log(2.0))
    ref.close(got[..., fine], want[..., fine], bound[..., fine])


@pytest.mark.parametrize("dtype,drop", [(F16, 20), (F16, 38), (BF16, 60)])
def test_attend_infinite_value_of_a_small_weight(dtype, drop):
    q, k, v, table, lens, lists, scale = sb.tail(dtype, drop, tokens=512)
    v[1, 0, 7, 9] = math.inf
    v[1, 0, 9, 10] = -math.inf
    got = run_attend(q.to(DEV), k.to(DEV), v.to(DEV), i32(table), i32(lens), i32(lists), scale)
    assert (got[..., 9] == math.inf).all() and (got[..., 10] == -math.inf).all()
    assert got[..., :9].isfinite().all() and got[..., 11:].isfinite().all()

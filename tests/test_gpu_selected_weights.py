"""The weights of the attention over selected pages: both 16-bit pieces of them, and their
range."""
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

"""paged_select_pages on bounds of very unequal sizes: the choice stays that of the 64-bit
scores, and pages that are listed anyway have no part in it."""
import math
import random

import pytest
import torch

import paged_kv_decode_16_gb300 as pkv
import selected_ref as ref
from test_gpu_selected import BF16, DEV, F16, check_select, i32, page_table, rand, status_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [50, 200, 400, 5000])
@pytest.mark.parametrize("far", [2.0 ** 50, -2.0 ** 50])
def test_select_beside_a_page_of_far_larger_keys(n, far):
    """One page whose bounds are 2^50 times the others', whose scores differ by less than a
    step of fp32: by multiples of 2^-14 at about 2000."""
    rng = random.Random(n)
    bounds = torch.full((n + 2, 1, 2, 64), 8.0, dtype=BF16)
    q = torch.full((1, 2, 64), 4.0, dtype=BF16)
    q[:, 1] = 0.0
    q[0, 0, 17] = 2.0 ** -7
    for p in range(n + 2):
        bounds[p, 0, :, 17] = rng.randrange(0, 60) * 2.0 ** -7
    table = page_table(rng, [16 * n], 16, n + 2, n)
    bounds[table[0][n // 3], 0, :, 5] = far
    if far < 0:
        q[0, 1] = -1.0  # (else the other head's score of the page, 0, is not far)
        bounds[table[0][n // 3], 0, :, 6] = -far * 8
    check_select(q.to(DEV), bounds.to(DEV), table, [16 * n], 16, min(37, n // 3), 1, 1)


@pytest.mark.parametrize("n", [50, 200, 5000])
def test_select_beside_a_page_of_ordinary_keys(n):
    """Pages whose products are below fp32's normal range, beside one of ordinary size."""
    gen = torch.Generator(device=DEV).manual_seed(n)
    rng = random.Random(n)
    table = page_table(rng, [16 * n], 16, n, n)
    q = rand(gen, 1, 3, 64, dtype=BF16) * 2.0 ** -45
    bounds = (rand(gen, n, 1, 2, 64, dtype=BF16) * 2.0 ** -100).sort(2).values
    bounds[table[0][n // 2]] = 2.0 ** 30
    bounds[table[0][n // 4]] = 0.0
    check_select(q, bounds, table, [16 * n], 16, n // 5, 1, 1)


@pytest.mark.parametrize("n,cols", [(40, 60), (120, 200), (200, 600)])
@pytest.mark.parametrize("first,last", [(1, 1), (3, 0), (0, 5)])
@pytest.mark.parametrize("x", [math.nan, math.inf, 2.0 ** 100])
def test_select_listed_pages_have_no_part_in_the_choice(n, cols, first, last, x):
    """Whatever the pages that are always listed hold, no score of another page is looked
    at a second time in 64 bits: their place in the workspace stays as it was."""
    gen = torch.Generator(device=DEV).manual_seed(n)
    rng = random.Random(n)
    table = page_table(rng, [16 * n], 16, n, cols)
    q = rand(gen, 1, 4, 64, dtype=BF16)
    bounds = rand(gen, n, 2, 2, 64, dtype=BF16).sort(2).values
    if first:
        bounds[table[0][first - 1], :, 1, 9] = x
    if last:
        bounds[table[0][n - last], :, 0, 8] = x
    sel = torch.full((1, 2, 12), 77, dtype=torch.int32, device=DEV)
    ws = pkv.alloc_select_workspace(1, 2, cols).fill_(165)
    st = status_word()
    pkv.paged_select_pages(q, bounds, i32(table), i32([16 * n]), 16, sel, ws, keep_first=first,
                           keep_last=last, dev_status=st)
    want, _ = ref.select(q, bounds, table, [16 * n], 16, 12, first, last)
    assert sel.tolist() == want and st.item() == 0
    assert (ws[:2 * cols * 8] == 165).all()


def test_select_flags_listed_pages_outside_the_pool():
    gen = torch.Generator(device=DEV).manual_seed(1)
    rng = random.Random(1)
    q = rand(gen, 1, 4, 64, dtype=F16)
    bounds = rand(gen, 90, 2, 2, 64, dtype=F16).sort(2).values
    for at in (0, 88, 89):
        table = page_table(rng, [16 * 90], 16, 90, 90)
        table[0][at] = 90
        assert check_select(q, bounds, table, [16 * 90], 16, 12, 1, 2) == ref.BAD_PAGE

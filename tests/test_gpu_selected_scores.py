"""paged_select_pages on bounds of very unequal sizes: the choice stays that of the 64-bit
scores."""
import random

import pytest
import torch

from test_gpu_selected import BF16, DEV, check_select, page_table, rand

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

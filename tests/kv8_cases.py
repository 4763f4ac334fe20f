"""Shapes of the 8-bit attention's accuracy tests, and their inputs."""
import numpy as np
import torch

import kv8_bound as kb

DECODE = [  # lens, Hq, Hkv, D, P
    ([1], 4, 2, 64, 16),
    ([37, 100], 4, 2, 64, 16),
    ([0, 1, 15, 16, 17, 0, 31, 32, 33, 250], 8, 2, 128, 16),
    ([500, 3, 77], 1, 1, 128, 32),
    ([300, 41], 7, 1, 128, 48),
    ([129, 64, 600], 12, 4, 64, 64),
    ([257, 90], 16, 1, 128, 256),
    ([160, 91], 24, 2, 64, 16),
    ([333, 5, 0], 24, 1, 64, 32),
    ([210, 18], 32, 1, 128, 16),
    ([1000], 33, 1, 128, 16),
    ([900, 1200, 40], 28, 4, 128, 32),
    ([50, 2000], 9, 3, 64, 128),
    ([2500, 2490], 128, 4, 64, 16),
    ([700], 64, 1, 128, 16),
    ([90, 1500, 0, 17], 96, 1, 64, 32),
    ([640, 33], 260, 2, 128, 48),
    ([1200] * 16 + [1111], 32, 1, 128, 16),
    ([3] * 40 + [9000] + [3] * 20, 8, 2, 128, 16),
    ([12000, 300], 4, 1, 64, 16),
]

MULTI = [  # Q, lens, Hq, Hkv, D, P
    (2, [1, 2, 3, 50, 0], 4, 2, 64, 16),
    (5, [5, 33, 300], 8, 2, 128, 32),
    (8, [200, 9, 3], 4, 1, 128, 16),
    (7, [64, 130], 7, 1, 64, 48),
    (16, [16, 400], 6, 3, 128, 16),
    (33, [33, 20, 210], 4, 2, 128, 64),
    (64, [64, 500, 10], 8, 2, 128, 16),
    (64, [128, 70], 3, 1, 64, 256),
    (3, [90, 1000], 32, 1, 128, 16),
    (40, [41, 700, 2, 0, 129], 4, 2, 128, 16),
    (64, [2000, 1], 5, 1, 64, 64),
    (17, [400, 18], 24, 3, 128, 48),
    (8, [1500, 900, 1211], 32, 8, 128, 16),
    (3, [1500, 700, 9, 1211, 900], 48, 8, 64, 32),
    (12, [800, 90], 8, 2, 128, 16),
    (7, [800, 90], 14, 2, 64, 16),
]

# batches about the largest whose ranges every CTA works out, and beyond
BATCHES = [(256, 6), (511, 4), (512, 140), (513, 4), (700, 140)]


def batch_lens(B):
    lens = np.random.default_rng(B).integers(0, 50, B)
    lens[-1] = 41
    return lens


def make(cache, lens, Q, Hq, Hkv, D, P, dtype, seed=40):
    """(the cache, poisoned where no row looks; q of dtype, on the host): rows whose
    results show which tokens they saw (kv8_bound.edges)."""
    c = cache(seed, lens, Hkv, D, P)
    q = np.random.default_rng(seed + 1).standard_normal((len(lens), Q, Hq, D))
    kb.edges(c, q, Q)
    return c.poison(), torch.from_numpy(q).to(dtype)

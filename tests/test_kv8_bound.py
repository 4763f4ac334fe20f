"""The attention's bound rejects what is wrong: zeros, the negated output, and a length
off by one, in every row of every shape of the accuracy tests."""
import numpy as np
import pytest
import torch

import kv8_bound as kb
import kv8_cases as cases
from test_gpu_kv8 import Cache

ALL = ([(1, *x) for x in cases.DECODE] + cases.MULTI
       + [(1, cases.batch_lens(B), Hq, 2, 64, 16) for B, Hq in cases.BATCHES])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Q,lens,Hq,Hkv,D,P", ALL)
def test_wrong_outputs_are_rejected(dtype, Q, lens, Hq, Hkv, D, P):
    c, q = cases.make(Cache, lens, Q, Hq, Hkv, D, P, dtype)
    qd, name = q.double().numpy(), str(dtype).split(".")[1]
    want, lim = kb.attention(qd, c.k, c.v, c.scales, c.table, c.lens, D ** -0.5, name)
    sees = (np.asarray(lens)[:, None] - Q + np.arange(Q) >= 0)  # [B][Q]: at least one token
    rejects = lambda out: (np.abs(out - want) > lim).any(-1)    # noqa: E731
    assert rejects(np.zeros_like(want))[sees].all()
    assert rejects(-want)[sees].all()
    # a query fewer than the tokens that it may see
    short = np.maximum(c.lens - 1, 0)
    off, _ = kb.attention(qd, c.k, c.v, c.scales, c.table, short, D ** -0.5, name)
    assert rejects(off)[sees].all()
    # and the exact output, rounded once, is not rejected
    assert not rejects(torch.from_numpy(want).to(dtype).double().numpy()).any()

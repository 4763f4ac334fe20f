"""The 8-bit attention against its 64-bit form, within a bound that rejects every wrong
row (kv8_bound, test_kv8_bound)."""
import pytest
import torch

import kv8_bound as kb
import kv8_cases as cases
import paged_kv_decode_16_gb300 as pkv
from test_gpu_kv8 import Cache, decode
from test_gpu_kv8_range import run

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("workers", [0, 1, 7])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P", cases.DECODE)
def test_decode(dtype, workers, lens, Hq, Hkv, D, P):
    c, q = cases.make(Cache, lens, 1, Hq, Hkv, D, P, dtype)
    c.gpu()
    out = decode(c, q[:, 0].cuda().contiguous(), D ** -0.5, workers)
    kb.check(c, q, out[:, None], D ** -0.5)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("workers", [0, 3])
@pytest.mark.parametrize("Q,lens,Hq,Hkv,D,P", cases.MULTI)
def test_multi(dtype, workers, Q, lens, Hq, Hkv, D, P):
    c, q = cases.make(Cache, lens, Q, Hq, Hkv, D, P, dtype)
    c.gpu()
    kb.check(c, q, run(c, q.cuda(), D ** -0.5, workers), D ** -0.5)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,Hq", cases.BATCHES)
def test_batches(dtype, B, Hq):
    c, q = cases.make(Cache, cases.batch_lens(B), 1, Hq, 2, 64, 16, dtype)
    c.gpu()
    out = decode(c, q[:, 0].cuda().contiguous(), 64 ** -0.5)
    kb.check(c, q, out[:, None], 64 ** -0.5)


def test_prompts_in_pieces():
    """Prompts appended in pieces of up to 64 tokens, each piece attended by its own
    queries, then steps: within the bound over the bytes that the appends left."""
    D, Hq, Hkv, P, Q = 64, 8, 2, 16, 64
    total = [150, 64, 7]
    c = Cache(42, total, Hkv, D, P, cap=[n + 3 for n in total])
    c.scales[:] = 255
    c.k[:] = c.v[:] = 0x7F
    c.gpu()
    pool = c.pool()
    gen = torch.Generator().manual_seed(8)
    mk = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    done = [0, 0, 0]
    while done != total:
        n = [min(Q, t - d) for t, d in zip(total, done)]
        seq = [b for b in range(3) for _ in range(n[b])]
        pos = [done[b] + i for b in range(3) for i in range(n[b])]
        q = mk(len(pos), Hq, D)
        rot = torch.empty_like(q)
        pkv.kv8_append_rope(pool, q, mk(len(pos), Hkv, D), mk(len(pos), Hkv, D), c.table_g,
                            i32(pos), 1e4, rot, i32(seq))
        done = [d + m for d, m in zip(done, n)]
        qs = torch.zeros(3, Q, Hq, D, dtype=torch.bfloat16, device="cuda")
        for b in range(3):
            if n[b]:
                qs[b, Q - n[b]:] = rot[i32(seq) == b]
        c.lens_g = i32(done)
        out = run(c, qs, D ** -0.5)
        c.k, c.v, c.scales = c.back()
        c.lens = c.lens_g.cpu().numpy()
        kb.check(c, qs, out, D ** -0.5)

"""The 8-bit step against append, then attention, on the paths that its other tests do not
take: many heads a KV head (the tensor-core tile, whose kernel starts beside the append)
and large batches (an append of more than one wave; above 512 sequences a plan kernel
behind it)."""
import numpy as np
import pytest
import torch

import kv8_bound as kb
import paged_kv_decode_16_gb300 as pkv
from test_gpu_kv8 import Cache, decode, i32, new_rows

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def pair(seed, lens, Hkv, D, P):
    return [Cache(seed, lens, Hkv, D, P).gpu() for _ in range(2)]


def check_step(dtype, lens, Hq, Hkv, D, P, theta, norm=False, exact=True):
    a, b = pair(50, lens, Hkv, D, P)
    B = len(lens)
    pos = np.asarray(lens) - 1
    kn, vn = new_rows(a, B, dtype)
    gen = torch.Generator().manual_seed(9)
    q = torch.randn(B, Hq, D, generator=gen).to(dtype).cuda()
    w = [(1 + 0.1 * torch.randn(D, generator=gen)).to(dtype).cuda() if norm else None
         for _ in range(2)]
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_kv8_workspace(B, Hq, Hkv, D)
    pkv.paged_decode_step_kv8(kn, vn, i32(pos), q, a.k_g, a.v_g, a.s_g, a.table_g, a.lens_g,
                              D ** -0.5, out, ws, rope_theta=theta, q_norm_weight=w[0],
                              k_norm_weight=w[1])
    assert pkv.pkv_read_device_status(ws) == 0
    rot = q
    if theta:
        rot = torch.empty_like(q)
        pkv.kv8_append_rope(b.pool(), q, kn, vn, b.table_g, i32(pos), theta, rot,
                            q_norm_weight=w[0], k_norm_weight=w[1])
    else:
        pkv.kv8_append(b.pool(), kn, vn, b.table_g, i32(pos))
    torch.cuda.synchronize()
    for x, y in zip(a.back(), b.back()):
        assert np.array_equal(x, y)
    assert torch.equal(out, decode(b, rot, D ** -0.5))
    assert (out[a.lens_g == 0] == 0).all()
    if exact:
        b.k, b.v, b.scales = b.back()
        kb.check(b, rot[:, None], out[:, None], D ** -0.5)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,P", [(64, 32), (128, 16)])
@pytest.mark.parametrize("theta,norm", [(0.0, False), (1e4, False), (5e5, True)])
def test_many_heads_a_kv_head(dtype, D, P, theta, norm):
    check_step(dtype, [700, 33, 0, 1, 256, 1500], 64, 1, D, P, theta, norm)


@pytest.mark.parametrize("Hq,Hkv", [(128, 2), (96, 1)])
def test_more_rows_than_a_tile(Hq, Hkv):
    check_step(BF, [90, 400], Hq, Hkv, 128, 48, 1e4)


@pytest.mark.parametrize("B", [300, 512, 600, 700])
@pytest.mark.parametrize("Hq,theta", [(4, 1e4), (128, 1e4), (4, 0.0)])
def test_large_batches(B, Hq, theta):
    lens = np.random.default_rng(B).integers(0, 60, B)
    lens[-2] = 900
    check_step(FP, lens, Hq, 2, 64, 16, theta, exact=B == 600)


@pytest.mark.parametrize("B,Hq", [(5, 8), (5, 128), (300, 8), (600, 8)])
def test_steps_in_a_row_without_a_wait(B, Hq):
    """Steps one behind another on one workspace, positions and lengths moved on by device
    copies between them: as with a wait behind each."""
    D, Hkv, steps = 128, 2, 6
    start = np.random.default_rng(B).integers(1, 40, B)
    start[0] = 333
    cap = start + steps
    a, b = (Cache(51, start, Hkv, D, 16, cap=cap).gpu() for _ in range(2))
    gen = torch.Generator().manual_seed(10)
    rows = [[torch.randn(B, h, D, generator=gen).bfloat16().cuda() for h in (Hkv, Hkv, Hq)]
            for _ in range(steps)]
    at = [i32(start + s) for s in range(steps + 1)]
    outs = []
    for c, wait in ((a, False), (b, True)):
        ws = pkv.alloc_kv8_workspace(B, Hq, Hkv, D)
        pos, ln = at[0].clone(), at[1].clone()
        out = [torch.empty(B, Hq, D, dtype=BF, device="cuda") for _ in range(steps)]
        torch.cuda.synchronize()
        for s in range(steps):
            pos.copy_(at[s])
            ln.copy_(at[s + 1])
            kn, vn, q = rows[s]
            pkv.paged_decode_step_kv8(kn, vn, pos, q, c.k_g, c.v_g, c.s_g, c.table_g, ln,
                                      D ** -0.5, out[s], ws, rope_theta=1e4)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert pkv.pkv_read_device_status(ws) == 0
        outs.append(out)
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    assert all(np.array_equal(x, y) for x, y in zip(a.back(), b.back()))

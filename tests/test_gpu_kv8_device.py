"""An 8-bit pool is used on its own device."""
import pytest
import torch

import paged_kv_decode_16_gb300 as pkv
from test_gpu_kv8 import Cache, i32, new_rows

pytestmark = pytest.mark.gpu


def test_append_to_a_pool_of_another_device():
    """Refused before anything is launched (the pool is made to say that its memory is on
    the next device)."""
    c = Cache(60, [20, 30], 2, 64, 16).gpu()
    kn, vn = new_rows(c, 2, torch.float16)
    q = torch.randn(2, 4, 64, device="cuda").half()
    before = [x.copy() for x in c.back()]
    for pool in (c.pool(), pkv.kv8_pool_create(c.NP, c.P, c.Hkv, c.D)):
        assert pool.device == torch.cuda.current_device()
        pool.device += 1
        with pytest.raises(ValueError, match="pool is on cuda"):
            pkv.kv8_append(pool, kn, vn, c.table_g, i32([0, 0]))
        with pytest.raises(ValueError, match="pool is on cuda"):
            pkv.kv8_append_rope(pool, q, kn, vn, c.table_g, i32([0, 0]), 1e4, q)
        pool.destroy()
    torch.cuda.synchronize()
    assert all((a == b).all() for a, b in zip(before, c.back()))

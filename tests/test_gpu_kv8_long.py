"""The 8-bit attention at the largest lengths that a table row can hold."""
import pytest
import torch

import paged_kv_decode_16_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq", [4, 64])  # the warp kernel; the tensor-core tile
@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 5000])
def test_lengths_to_the_end_of_32_bits(n, Hq):
    """Every page of the row is page 1, whose keys are zeros and values ones; the last token's
    block is read up to it only: page 0, NaN, is the row's last where it is not full."""
    P, D = 256, 64
    k = torch.zeros(2, 1, P, D, dtype=torch.uint8, device="cuda")
    v = torch.full((2, 1, P, D), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    last = n % P
    v[0, 0, last:] = 0x7F  # behind the end
    s = torch.full((2, 1, P // 16, 2), 127, dtype=torch.uint8, device="cuda")
    table = torch.ones(1, 2 ** 31 // P, dtype=torch.int32, device="cuda")
    table[0, n // P] = 0 if last else 1
    q = torch.randn(1, Hq, D, device="cuda").bfloat16()
    out = torch.full_like(q, float("nan"))
    ws = pkv.alloc_kv8_workspace(1, Hq, 1, D)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    e4m3 = torch.float8_e4m3fn
    pkv.paged_decode_attention_kv8(q, k.view(e4m3), v.view(e4m3), s, table, lens, D ** -0.5, out, ws)
    assert pkv.pkv_read_device_status(ws) == 0
    # equal weights of ones: sums of whole numbers below 2^24 a worker, exact; the merges
    # round by 2^-24 each, a few thousand of them
    assert (out - 1).abs().max() <= 2.0 ** -8

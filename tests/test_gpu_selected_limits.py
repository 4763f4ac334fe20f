"""paged_tables_build and kv_page_bounds at the ends of their documented ranges."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BATCHES = """
import sys, torch
sys.path.insert(0, {root!r})
import paged_kv_decode_16_gb300 as pkv
DEV, N = "cuda", int(sys.argv[1])
for B in map(int, sys.argv[2:]):
    i32 = lambda n, x: torch.full((n,), x, dtype=torch.int32, device=DEV)
    free = torch.randperm(B, device=DEV).to(torch.int32)
    table, lens, starts = i32(2 * B, -1).view(B, 2), i32(B, 7), i32(B + 1, 7)
    pos, seq, end, st = i32(N, 7), i32(N, 7), i32(1, 7), i32(1, 0)
    slots = torch.full((N,), 7, dtype=torch.int64, device=DEV)
    pkv.paged_tables_build(i32(B, 0), i32(B, 1), free, None, end, table, 16, B, lens, starts,
                           pos, seq, slots, dev_status=st)
    assert st.item() == 0 and end.item() == B and (lens == 1).all()
    assert torch.equal(starts, torch.arange(B + 1, dtype=torch.int32, device=DEV))
    assert torch.equal(slots[:B], free.long() * 16) and (slots[B:] == -1).all()
    assert torch.equal(table[:, 0], free) and (table[:, 1] == -1).all()
    assert torch.equal(seq[:B], torch.arange(B, dtype=torch.int32, device=DEV))
    assert (seq[B:] == -1).all() and (pos[:B] == 0).all() and (pos[B:] == -1).all()
print("done")
"""


@pytest.mark.parametrize("tokens", [5000, 8400000])  # sums in 32 and in 64 bits
def test_tables_of_batches_about_the_default_shared_memory(tokens):
    """12 bytes a request reach the 48 KB of shared memory that a launch has unasked, which
    its static part shares, at about 4090 requests.  In a process of its own, the smaller
    batches first: a limit that a larger batch raised stays raised."""
    r = subprocess.run([sys.executable, "-c", BATCHES.format(root=ROOT), str(tokens),
                        *map(str, (4072, 4073, 4074, 4083, 4084, 4090, 4095, 4096, 4500))],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr

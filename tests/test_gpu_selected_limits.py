"""paged_tables_build and kv_page_bounds at the ends of their documented ranges."""
import os
import subprocess
import sys

import pytest
import torch

import paged_kv_decode_16_gb300 as pkv
from test_gpu_selected import DEV, i32, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory_back():
    """The largest tests take tens of GB: not kept for the tests behind them."""
    yield
    torch.cuda.empty_cache()


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


def same(x, first, want, step=1 << 26):
    """x[i] == want(i) for i from `first` on, in pieces."""
    for a in range(first, x.numel(), step):
        i = torch.arange(a, min(a + step, x.numel()), device=DEV)
        if not torch.equal(x[a:a + step].long(), want(i)):
            return False
    return True


def test_tables_of_the_most_token_rows():
    """2^31 - 1 rows: a row's number plus a stride of the grid is beyond 32 bits."""
    N, page = 2 ** 31 - 1, 256
    new = [3, N - 100 - 3]
    need = [1, -(-new[1] // page)]
    free = torch.randperm(sum(need), device=DEV).to(torch.int32)
    table = torch.full((2, need[1]), -1, dtype=torch.int32, device=DEV)
    lens, starts, end, st = i32([0, 0]), i32([0] * 3), i32([0]), status_word()
    pos, seq = (torch.full((N,), 7, dtype=torch.int32, device=DEV) for _ in range(2))
    slots = torch.full((N,), 7, dtype=torch.int64, device=DEV)
    pkv.paged_tables_build(i32([0, 0]), i32(new), free, None, end, table, page, sum(need), lens,
                           starts, pos, seq, slots, dev_status=st)
    assert st.item() == 0 and end.item() == sum(need)
    assert lens.tolist() == new and starts.tolist() == [0, 3, N - 100]
    assert torch.equal(table[1], free[1:]) and table[0, 0] == free[0]
    assert (table[0, 1:] == -1).all()
    pages = free.long()
    assert pos[:3].tolist() == [0, 1, 2] and (seq[:3] == 0).all()
    assert torch.equal(slots[:3], pages[0] * page + torch.arange(3, device=DEV))
    none = N - 100
    assert same(seq[:none], 3, torch.ones_like)
    assert same(pos[:none], 3, lambda i: i - 3)
    assert same(slots[:none], 3, lambda i: pages[1 + (i - 3) // page] * page + (i - 3) % page)
    for x in (pos, seq, slots):
        assert (x[none:] == -1).all()


def test_bounds_of_the_most_slots():
    """2^31 - 1 slots, of which the last ones, and those around a tile's ends, hold rows."""
    N, NP, page, hkv, d = 2 ** 31 - 1, 90, 16, 2, 64
    gen = torch.Generator(device=DEV).manual_seed(1)
    k_pool = torch.randn(NP, hkv, page, d, generator=gen, device=DEV).to(torch.bfloat16)
    pool = pkv.kv_pool_create(NP, page, hkv, d, torch.bfloat16, k_pool, torch.empty_like(k_pool))
    slots = torch.full((N,), -1, dtype=torch.int64, device=DEV)
    pages = torch.randperm(NP, generator=gen, device=DEV)
    at = torch.arange(NP, device=DEV) % page
    slots[N - 80:] = (pages * page + at)[10:]      # a page each
    slots[:10] = (pages * page + at)[:10]
    bounds = torch.full((NP, hkv, 2, d), 55.0, dtype=torch.bfloat16, device=DEV)
    st = status_word()
    pkv.kv_page_bounds(pool, slots, bounds, dev_status=st)
    assert st.item() == 0
    for p, x in zip(pages.tolist(), at.tolist()):
        rows = k_pool[p, :, :x + 1]
        assert torch.equal(bounds[p, :, 0], rows.amin(1))
        assert torch.equal(bounds[p, :, 1], rows.amax(1))


def test_select_into_the_longest_list():
    """max_pages 2^31 - 1: every page is listed, -1 behind them to the list's end."""
    K, n = 2 ** 31 - 1, 700
    sel = torch.full((1, 1, K), 7, dtype=torch.int32, device=DEV)
    q = torch.ones(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    bounds = torch.ones(n, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.arange(n, dtype=torch.int32, device=DEV)[None]
    st = status_word()
    for cols, ws in ((n, pkv.alloc_select_workspace(1, 1, n)),       # two launches
                     (200, pkv.alloc_select_workspace(1, 1, 200))):  # one
        sel.fill_(7)
        pkv.paged_select_pages(q, bounds, table[:, :cols].contiguous(), i32([16 * cols - 3]), 16,
                               sel, ws, dev_status=st)
        assert st.item() == 0
        assert torch.equal(sel[0, 0, :cols].long(), torch.arange(cols, device=DEV))
        assert (sel[0, 0, cols:] == -1).all()

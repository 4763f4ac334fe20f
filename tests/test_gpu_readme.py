"""The README's step with selected pages, run as it is printed."""
import os
import textwrap

import pytest
import torch

import paged_kv_decode_16_gb300 as pkv
import selected_ref as ref
from test_gpu_selected import BF16, DEV, i32, i64, rand

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def block():
    lines = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read().splitlines()
    first = next(i for i, s in enumerate(lines) if "a step that attends to selected pages:" in s)
    last = first
    while lines[last].startswith("    "):
        last += 1
    return textwrap.dedent("\n".join(lines[first:last]))


def test_readme_step_with_selected_pages():
    """Each request's last new token, rotated, is what selects and attends."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    B, Hq, Hkv, D, P, num_pages, cols = 3, 8, 2, 128, 16, 300, 120
    new = [1700, 3, 200]
    n = sum(new)
    k_pool, v_pool = (torch.zeros(num_pages, Hkv, P, D, dtype=BF16, device=DEV) for _ in range(2))
    ns = dict(pkv=pkv, torch=torch, B=B, Hq=Hq, Hkv=Hkv, D=D, P=P, num_pages=num_pages,
              k_pool=k_pool, v_pool=v_pool, cached_lens=i32([0] * B), new_lens=i32(new),
              free_pages=i32(list(range(num_pages))[::-1]), free_begin=i32([0]),
              free_end=i32([0]), page_table=torch.full((B, cols), -1, dtype=torch.int32, device=DEV),
              context_lens=i32([0] * B), query_starts=i32([0] * (B + 1)), positions=i32([0] * n),
              seq_ids=i32([0] * n), slots=i64([0] * n),
              qkv=rand(gen, n, Hq + 2 * Hkv, D, dtype=BF16),
              q_rot=torch.zeros(n, Hq, D, dtype=BF16, device=DEV),
              # of the README's examples above it
              q=rand(gen, B, Hq, D, dtype=BF16), out=torch.zeros(B, Hq, D, dtype=BF16, device=DEV))
    exec(compile(block(), "README.md", "exec"), ns)
    last = torch.tensor(new).cumsum(0) - 1
    # the rotation of the query rows that count, then the rest on what they are
    q = ns["qkv"][:, :Hq]
    y, err = ref.turned(q[last], torch.tensor(new) - 1,
                        ref.frequencies(D, 500000.0, "turns", 8.0, 1.0, 4.0, 8192.0), False)
    asked = ns["q_rot"][last]
    ref.close(asked, y, ref.rounded(y, err, BF16))
    table = ns["page_table"].tolist()
    lists, _ = ref.select(asked, ns["bounds"], table, new, P, 64, 1, 2)
    assert ns["selected"].tolist() == lists
    ref.close(ns["out"], *ref.attend(asked, k_pool, v_pool, table, new, lists, D ** -0.5))

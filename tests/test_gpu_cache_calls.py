"""Calls of the decoding operators that their documentation allows and that ordinary use meets rarely: first calls of
a process, several threads, empty problems, pointers between others."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import lsh_attention_hash_b200 as lsh
from oracle import cache_oracle as co
from tests.test_gpu_cache import DEV, Cache, _status, np64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _wide_select(pages):
    """The choice of 2 of ``pages`` pages of 64 tokens, 4 rounds (scored by the scoring kernel): page 5 has hits."""
    tags = torch.zeros(2, 1, 4, 64, dtype=torch.int16, device=DEV)
    tags[1] = 9
    table = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
    table[0, 5] = 1
    qb = torch.full((1, 1, 4, 1), 9, dtype=torch.int32, device=DEV)
    ctx = torch.tensor([pages * 64], dtype=torch.int32, device=DEV)
    return lambda: lsh.lsh_cache_select(tags, qb, table, ctx, 2)[0]


FIRST = """
import sys
sys.path.insert(0, {root!r})
from tests.test_gpu_cache_calls import _wide_select
for pages in {pages!r}:
    assert _wide_select(pages)().flatten().tolist() == [5, pages - 1], pages
print("fine")
"""


@pytest.mark.parametrize("pages", [(12160,), (12220,), (12221,), (12288,), (12289,), (49152, 12230, 100)])
def test_select_of_any_width_as_the_first_call(pages):
    """Scores of 12288 pages are 48 KB of shared memory, to which the kernel's own variables come."""
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, pages=pages)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout == "fine\n", r.stderr[-2000:]


def test_selects_of_several_threads():
    """Calls with tables of different widths at once: none lowers what another one's launch needs."""
    widths = [12300, 49152, 20000, 40000]
    calls, wrong = [_wide_select(w) for w in widths], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    got = calls[i]()
                if got.flatten().tolist() != [5, widths[i] - 1]:
                    wrong.append((i, got))
        except Exception as e:  # (reported by the test's thread)
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(widths))]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and _status() == 0

"""The planners at their largest sizes, each in a process that has made no larger call before: the shared memory that a
kernel may have is set once for a process, so that a larger call hides what a smaller one lacks. Whole numbers: every
comparison is for equality."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import pages as OP

pytestmark = pytest.mark.gpu

P, M = 16, 2


def state(rows, num_pages):
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, M * P // 2 + 1, rows).astype(np.int32)
    table = np.full((rows, M), -1, dtype=np.int32)
    perm = rng.permutation(num_pages).astype(np.int32)
    held = -(-lens // P)
    for j in range(M):
        live = held > j
        table[live, j] = perm[np.arange(rows)[live] * M + j]
    return table, lens, OP.counts(table, lens, num_pages, P).astype(np.int32), rng


def run_resize(rows):
    from load_balanced_split_step_b200 import binding as B
    table, lens, ref, rng = state(rows, rows * M)
    new = np.clip(lens + rng.integers(-P, P, rows), 0, M * P).astype(np.int32)
    want = OP.resize(table, lens, new, ref, P)
    t, o, n, c = (torch.from_numpy(a).cuda() for a in (table, lens, new, ref))
    up = B.resize_pages(t, o, n, c, P)
    assert want is not None and int(up.status.item()) == 0
    assert np.array_equal(up.block_table.cpu().numpy(), want[0]) and np.array_equal(up.ref_count.cpu().numpy(), want[1])


def run_fork(rows):
    from load_balanced_split_step_b200 import binding as B
    table, lens, ref, rng = state(rows, rows * M)
    par = rng.integers(-1, rows, rows).astype(np.int32)
    want = OP.fork(table, lens, ref, par, P)
    t, l, c, p = (torch.from_numpy(a).cuda() for a in (table, lens, ref, par))
    up = B.fork_pages(t, l, c, p, P)
    assert want is not None and int(up.status.item()) == 0
    assert np.array_equal(up.block_table.cpu().numpy(), want[0]) and np.array_equal(up.ref_count.cpu().numpy(), want[2])
    assert np.array_equal(up.seq_lens.cpu().numpy(), want[1])


# Rows whose needs take just under 48 KB of shared memory (8 bytes a row in a resize, 12 in a fork), exactly 48, and most.
@pytest.mark.parametrize("what,rows", [("resize", 6092), ("resize", 6100), ("resize", 6144), ("resize", 6145),
                                       ("resize", 8192), ("fork", 4061), ("fork", 4070), ("fork", 4096), ("fork", 4097),
                                       ("fork", 8192)])
def test_large_batches_in_a_process_of_their_own(what, rows):
    code = f"from tests.test_gpu_pages_limits import run_{what}; run_{what}({rows})"
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]

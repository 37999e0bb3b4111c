"""Launches that the runtime refuses: they raise, leave nothing behind, and no call runs twice. The refusal is made on the
host: a launch into a stream whose capture has been invalidated. Page updates are whole numbers, compared for equality
with the oracle."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import pages as OP
from tests.test_gpu_pages import dev, moves_of, same, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def refused_launch(B):
    """A call that fails at its launch, and is caught."""
    cuda = ctypes.CDLL("libcuda.so.1")
    s = torch.cuda.Stream()
    cache = torch.zeros((4, 16), dtype=torch.uint8, device="cuda")
    moves = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    n, st = torch.zeros(1, dtype=torch.int32, device="cuda"), B.new_status("cuda")
    torch.cuda.synchronize()
    handle, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
    assert cuda.cuStreamBeginCapture_v2(handle, 1) == 0  # of this thread
    try:
        assert cuda.cuStreamSynchronize(handle) != 0  # not allowed in a capture, and the end of this one
        with torch.cuda.stream(s), pytest.raises(B.HpcError, match="CUDA error"):
            B.copy_pages([cache], moves, n, status=st)
    finally:
        cuda.cuStreamEndCapture(handle, ctypes.byref(graph))
    assert not graph.value


@pytest.mark.parametrize("short", [True, False])
def test_an_update_after_a_refused_launch_runs_once(B, monkeypatch, short):
    if not short:
        monkeypatch.setattr(B, "_fast", None)
    rows, M, N, P = 20, 9, 300, 16
    table, lens, ref = state(3, rows, M, N, P, 100, share=True)
    new = np.minimum(lens + 20, M * P).astype(np.int32)
    want = OP.resize(table, lens, new, ref, P)
    t, o, n, c = dev(table, lens, new, ref)
    refused_launch(B)
    up = B.resize_pages(t, o, n, c, P, block_table_out=t, ref_count_out=c)
    assert int(up.status.item()) == 0 and moves_of(up) == want[2]
    same(t, want[0])
    same(c, want[1])
    want = OP.compact(want[0], want[1])
    refused_launch(B)
    up = B.compact_pages(t, c, block_table_out=t, ref_count_out=c)
    assert int(up.status.item()) == 0 and moves_of(up) == want[3] and want[3]
    same(t, want[0])
    same(c, want[1])
    same(up.page_map, want[2])

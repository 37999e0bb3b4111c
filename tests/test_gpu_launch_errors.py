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


def test_a_launch_that_fails_is_not_tried_again(B, monkeypatch):
    """The short way with a library whose resize reports a failed launch: the long way must not run it again."""
    assert B._fast is not None
    tried = []

    class Library:
        def __getattr__(self, name):
            if name.startswith("hpc_pages"):
                tried.append(name)
            return getattr(lib, name)

    lib, resize = B._lib, B._lib.hpc_pages_resize
    fake = ctypes.CFUNCTYPE(ctypes.c_int, *resize.argtypes)(lambda *a: tried.append("short") or B.HPC_ERR_CUDA)
    at = [ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in B._FAST_CALLS]
    at[B._FAST_CALLS.index("hpc_pages_resize")] = ctypes.cast(fake, ctypes.c_void_p).value
    t, o, n, c = dev(*(np.zeros(s, dtype=np.int32) for s in ((2, 3), 2, 2, 5)))
    monkeypatch.setattr(B, "_lib", Library())
    try:
        B._fast.bind(B._check, *at)
        with pytest.raises(B.HpcError, match="hpc_pages_resize: CUDA error"):
            B.resize_pages(t, o, n, c, 16)
    finally:
        B._bind(lib)
    assert tried == ["short"]

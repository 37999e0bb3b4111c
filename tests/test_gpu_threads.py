"""The short way in from several Python threads."""
import threading
import time

import pytest
import torch

from oracle import pages as OP
from tests.test_gpu_pages import dev, moves_of, same, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    assert binding._fast is not None
    return binding


def test_other_threads_run_while_a_launch_waits(B):
    """A stream that is held up for about a second takes some thousand launches; the next one waits, and the
    interpreter is not kept from the other threads meanwhile."""
    table, ref = dev(*state(1, 4, 5, 33, 16, 70)[::2])
    bufs = dict(block_table_out=table.clone(), ref_count_out=ref.clone(), page_map=ref.clone(), n_moves=ref[:1].clone(),
                moves=torch.zeros((33, 2), dtype=torch.int32, device="cuda"), status=B.new_status("cuda"))
    B.compact_pages(table, ref, **bufs)
    torch.cuda.synchronize()
    gaps, stop = [0.0], threading.Event()

    def watch():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.002)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    t = threading.Thread(target=watch)
    t.start()
    torch.cuda._sleep(2_000_000_000)
    begun = time.perf_counter()
    for _ in range(4000):
        B.compact_pages(table, ref, **bufs)
    spent = time.perf_counter() - begun
    stop.set()
    t.join()
    torch.cuda.synchronize()
    assert spent > 0.5  # the queue was full, or the case shows nothing
    assert max(gaps) < 0.3, max(gaps)
    assert int(bufs["status"].item()) == 0


def test_threads_get_their_own_results(B):
    """Four threads, each with a stream and a state of its own, whose calls need new status words time and again."""
    failed = []

    def work(seed):
        try:
            rows, M, N, P = 5 + seed, 9, 300, 16
            table, lens, ref = state(seed, rows, M, N, P, 60)
            new = (lens + 20).astype(lens.dtype)
            want = OP.resize(table, lens, new, ref, P)
            with torch.cuda.stream(torch.cuda.Stream()):
                t, o, n, c = dev(table, lens, new, ref)
                ups = [B.resize_pages(t, o, n, c, P) for _ in range(400)]
                torch.cuda.current_stream().synchronize()
                assert len({u.status.data_ptr() for u in ups}) == 400
                for u in ups[::40]:
                    assert int(u.status.item()) == 0 and moves_of(u) == want[2]
                    same(u.block_table, want[0])
                    same(u.ref_count, want[1])
        except BaseException as e:  # noqa: BLE001 (reported by the test's own thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[0]

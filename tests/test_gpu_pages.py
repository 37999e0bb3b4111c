"""Cache upkeep on the GPU (resize, fork, compact, page copies) against the request-by-request oracle.
Everything is whole numbers or bytes, so every comparison is for equality."""
import numpy as np
import pytest
import torch

from oracle import pages as OP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def state(seed, rows, max_pages, num_pages, P, max_len, share=False, empty=0.2):
    """(table, lens, ref) over a scattered pool; with `share`, odd rows start with pages of the row before."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, max_len + 1, rows)
    lens[rng.random(rows) < empty] = 0
    perm = rng.permutation(num_pages)
    table = np.full((rows, max_pages), -1, dtype=np.int32)
    o = 0
    for r, n in enumerate(lens):
        h = OP.held(n, P)
        table[r, :h] = perm[o:o + h]
        o += h
    assert o <= num_pages
    if share:
        for r in range(1, rows, 2):
            k = min(OP.held(lens[r - 1], P), OP.held(lens[r], P))
            k = int(rng.integers(0, k + 1))
            table[r, :k] = table[r - 1, :k]
    return table, lens.astype(np.int32), OP.counts(table, lens, num_pages, P).astype(np.int32)


def dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def moves_of(up):
    n = int(up.n_moves.item())
    return [tuple(m) for m in up.moves[:n].cpu().tolist()]


def same(t, a):
    assert np.array_equal(t.cpu().numpy(), np.asarray(a))


SHAPES = [  # rows, max_pages, num_pages, page_size, max_len
    (1, 1, 1, 16, 16), (1, 3, 40, 1, 3), (4, 5, 33, 16, 70), (37, 9, 777, 32, 280), (256, 70, 20011, 64, 4400),
    (1025, 4, 8192, 128, 500), (5, 300, 260000, 16, 4790),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_resize(B, shape, share, inplace):
    rows, M, N, P, max_len = shape
    table, lens, ref = state(rows + P + share, rows, M, N, P, max_len, share)
    rng = np.random.default_rng(7)
    new = np.clip(lens + rng.integers(-2 * P, 2 * P + 1, rows), 0, M * P).astype(np.int32)
    new[rng.random(rows) < 0.2] = 0
    want = OP.resize(table, lens, new, ref, P)
    t, o, n, c = dev(table, lens, new, ref)
    up = B.resize_pages(t, o, n, c, P, block_table_out=t if inplace else None, ref_count_out=c if inplace else None)
    if want is None:
        assert int(up.status.item()) == B.DEV_STATUS["capacity"] and moves_of(up) == []
        same(up.block_table, table)
        same(up.ref_count, ref)
        return
    assert int(up.status.item()) == 0
    same(up.block_table, want[0])
    same(up.ref_count, want[1])
    assert moves_of(up) == want[2]
    if not inplace:
        same(t, table)
        same(c, ref)
    if not share:
        assert np.array_equal(want[1], OP.counts(want[0], new, N, P))


@pytest.mark.parametrize("N,taken", [(70000, 0.97), (150000, 0.5), (65537, 0.999)])
def test_a_crowded_large_pool(B, N, taken):
    """Most pages are held elsewhere, so that the pages that are taken lie far apart, in every part of a warp's run."""
    rng = np.random.default_rng(N)
    rows, M, P = 60, 40, 16
    ref = (rng.random(N) < taken).astype(np.int32)
    table = np.full((rows, M), -1, dtype=np.int32)
    lens = rng.integers(1, M * P // 2, rows).astype(np.int32)
    held = rng.permutation(np.flatnonzero(ref == 0))
    o = 0
    for r, n in enumerate(lens):
        h = min(OP.held(n, P), max(1, (len(held) - o) // (2 * (rows - r))))
        lens[r] = min(n, h * P)
        table[r, :h] = held[o:o + h]
        ref[held[o:o + h]] = 1
        o += h
    free = int((ref == 0).sum())
    new = np.minimum(lens + rng.integers(0, max(2, free * P // rows), rows), M * P).astype(np.int32)
    t, l, n, c = dev(table, lens, new, ref)
    want = OP.resize(table, lens, new, ref, P)
    up = B.resize_pages(t, l, n, c, P)
    assert int(up.status.item()) == (B.DEV_STATUS["capacity"] if want is None else 0)
    if want is None:
        same(up.block_table, table)
        same(up.ref_count, ref)
    else:
        same(up.block_table, want[0])
        same(up.ref_count, want[1])
        par = rng.integers(0, rows, rows).astype(np.int32)
        want = OP.fork(want[0], new, want[1], par, P)
        up = B.fork_pages(up.block_table, n, up.ref_count, dev(par)[0], P)
        assert int(up.status.item()) == (B.DEV_STATUS["capacity"] if want is None else 0)
        if want is not None:
            same(up.block_table, want[0])
            same(up.ref_count, want[2])
            assert moves_of(up) == want[3]
    want = OP.compact(table, ref)
    up = B.compact_pages(t, c)
    same(up.block_table, want[0])
    same(up.ref_count, want[1])
    assert moves_of(up) == want[3]


def test_resize_copies_a_shared_part_filled_page_on_write(B):
    """Both sharers of a part-filled page grow in one call: each takes a copy, the page itself is left
    free, and it is not taken in the same call."""
    P = 16
    table = np.array([[3, 0, -1], [3, 0, -1], [1, -1, -1]], dtype=np.int32)
    lens = np.array([20, 20, 5], dtype=np.int32)
    ref = np.array([2, 1, 0, 2, 0, 0], dtype=np.int32)
    new = np.array([21, 33, 5], dtype=np.int32)
    t, o, n, c = dev(table, lens, new, ref)
    up = B.resize_pages(t, o, n, c, P)
    same(up.block_table, [[3, 2, -1], [3, 4, 5], [1, -1, -1]])
    same(up.ref_count, [0, 1, 1, 2, 1, 1])
    assert moves_of(up) == [(0, 2), (0, 4)]


def test_resize_with_too_few_pages_changes_nothing(B):
    table, lens, ref = state(5, 6, 8, 20, 16, 40, empty=0)
    new = np.full(6, 128, dtype=np.int32)
    assert OP.resize(table, lens, new, ref, 16) is None
    for inplace in (False, True):
        t, o, n, c = dev(table, lens, new, ref)
        up = B.resize_pages(t, o, n, c, 16, block_table_out=t if inplace else None,
                            ref_count_out=c if inplace else None)
        assert int(up.status.item()) == B.DEV_STATUS["capacity"]
        assert int(up.n_moves.item()) == 0
        same(up.block_table, table)
        same(up.ref_count, ref)


def test_resize_flags_bad_rows_and_leaves_them(B):
    P = 16
    table = np.array([[0, 1, 9], [2, 3, -1], [4, -1, -1], [77, -1, -1]], dtype=np.int32)
    lens = np.array([-1, 32, 16, 10], dtype=np.int32)
    new = np.array([5, 49, 17, 0], dtype=np.int32)  # row 1: beyond the table; row 3: releases a page outside the pool
    ref = np.array([1, 1, 1, 1, 1, 0, 0, 0, 0, 1], dtype=np.int32)
    t, o, n, c = dev(table, lens, new, ref)
    up = B.resize_pages(t, o, n, c, P)
    assert int(up.status.item()) == B.DEV_STATUS["bad_seqlen"] | B.DEV_STATUS["bad_page"]
    same(up.block_table, [[0, 1, 9], [2, 3, -1], [4, 5, -1], [-1, -1, -1]])
    same(up.ref_count, [1, 1, 1, 1, 1, 1, 0, 0, 0, 1])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["reorder", "one", "drop", "wider"])
def test_fork(B, shape, kind):
    rows, M, N, P, max_len = shape
    table, lens, ref = state(rows * 3 + P, rows, M, N, P, max_len)
    rng = np.random.default_rng(11)
    par = {"reorder": rng.integers(0, rows, rows), "one": np.full(rows, rows // 2), "drop": rng.integers(-1, rows, rows),
           "wider": np.arange(3 * rows) // 3}[kind].astype(np.int32)
    want = OP.fork(table, lens, ref, par, P)
    t, l, c, p = dev(table, lens, ref, par)
    up = B.fork_pages(t, l, c, p, P)
    if want is None:
        assert int(up.status.item()) == B.DEV_STATUS["capacity"] and moves_of(up) == []
        same(up.ref_count, ref)
        assert int(up.block_table.max().item()) == -1 and int(up.seq_lens.abs().max().item()) == 0
        return
    assert int(up.status.item()) == 0
    same(up.block_table, want[0])
    same(up.seq_lens, want[1])
    same(up.ref_count, want[2])
    assert moves_of(up) == want[3]
    assert np.array_equal(want[2], OP.counts(want[0], want[1], N, P))


def test_fork_counts_in_place_and_bad_parents(B):
    P = 16
    table = np.array([[0, 1], [2, -1]], dtype=np.int32)
    lens = np.array([20, 99], dtype=np.int32)  # row 1: beyond the table
    ref = np.array([1, 1, 1, 0, 0], dtype=np.int32)
    par = np.array([0, 5, 1, 0, -1, -2], dtype=np.int32)
    t, l, c, p = dev(table, lens, ref, par)
    up = B.fork_pages(t, l, c, p, P, ref_count_out=c)
    assert int(up.status.item()) == B.DEV_STATUS["bad_index"] | B.DEV_STATUS["bad_seqlen"]
    same(up.block_table, [[0, 1], [-1, -1], [-1, -1], [0, 3], [-1, -1], [-1, -1]])
    same(up.seq_lens, [20, 0, 0, 20, 0, 0])
    same(up.ref_count, [2, 1, 1, 1, 0])
    assert up.ref_count is c and moves_of(up) == [(1, 3)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("inplace", [False, True])
def test_compact(B, shape, inplace):
    rows, M, N, P, max_len = shape
    table, lens, ref = state(rows * 5 + P, rows, M, N, P, max_len, share=True)
    ref[N // 2] += 3  # held outside the table too
    want = OP.compact(table, ref)
    t, c = dev(table, ref)
    up = B.compact_pages(t, c, block_table_out=t if inplace else None, ref_count_out=c if inplace else None)
    assert int(up.status.item()) == 0
    same(up.block_table, want[0])
    same(up.ref_count, want[1])
    same(up.page_map, want[2])
    assert moves_of(up) == want[3]
    n = int((ref > 0).sum())
    assert (want[1][:n] > 0).all() and (want[1][n:] == 0).all()


def test_compact_renames_stale_entries(B):
    t, c = dev(np.array([[4, 1, 9, -7]], dtype=np.int32), np.array([0, 0, 0, 0, 2], dtype=np.int32))
    up = B.compact_pages(t, c)
    assert int(up.status.item()) == B.DEV_STATUS["bad_page"]
    same(up.block_table, [[0, -1, -1, -1]])
    same(up.ref_count, [2, 0, 0, 0, 0])
    same(up.page_map, [-1, -1, -1, -1, 0])


@pytest.mark.parametrize("shape,dtype,layers", [
    ((50, 2, 16, 64), torch.bfloat16, 2), ((9, 8, 64, 128), torch.float8_e4m3fn, 1), ((7, 1, 1, 16), torch.uint8, 3),
    ((11, 3, 5, 8), torch.bfloat16, 1), ((300, 1, 16, 64), torch.bfloat16, 130),
])
def test_copy_pages(B, shape, dtype, layers):
    N = shape[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    caches = [torch.randint(0, 256, (*shape[:-1], shape[-1] * dtype.itemsize), generator=g, device="cuda",
                            dtype=torch.uint8).view(dtype) for _ in range(2 * layers)]
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(4))
    k = N // 2
    src, dst = perm[:k], perm[k:2 * k]
    moves = torch.full((N, 2), 12345, dtype=torch.int32)
    moves[:k, 0], moves[:k, 1] = src, dst
    want = [c.clone() for c in caches]
    for w in want:
        w.view(torch.uint8)[dst.cuda()] = w.view(torch.uint8)[src.cuda()]
    st = B.copy_pages(caches, moves.cuda(), torch.tensor([k], dtype=torch.int32, device="cuda"))
    assert int(st.item()) == 0
    for c, w in zip(caches, want):
        assert torch.equal(c.view(torch.uint8), w.view(torch.uint8))


def test_copy_pages_flags(B):
    cache = torch.arange(4 * 16, dtype=torch.uint8, device="cuda").reshape(4, 16)
    before = cache.clone()
    moves = torch.tensor([[0, 9], [-1, 2], [1, 3]], dtype=torch.int32, device="cuda")
    st = B.copy_pages([cache], moves, torch.tensor([3], dtype=torch.int32, device="cuda"))
    assert int(st.item()) == B.DEV_STATUS["bad_page"]
    assert torch.equal(cache[:3], before[:3]) and torch.equal(cache[3], before[1])
    st = B.copy_pages([cache], moves[2:], torch.tensor([7], dtype=torch.int32, device="cuda"))
    assert int(st.item()) == B.DEV_STATUS["capacity"]
    st = B.copy_pages([cache], moves, torch.tensor([-2], dtype=torch.int32, device="cuda"))
    assert int(st.item()) == B.DEV_STATUS["capacity"]


def test_updates_are_captured_and_replayed(B):
    """A captured grow + fork + copy on a side stream, replayed on new lengths."""
    P, N, M = 16, 400, 12
    table, lens, ref = state(21, 16, M, N, P, 90)
    t, l, c = dev(table, lens, ref)
    new = torch.clamp(l + 3, max=M * P)
    par = torch.arange(16, dtype=torch.int32, device="cuda") // 2
    cache = torch.randint(0, 256, (N, 32), device="cuda", dtype=torch.uint8)
    bufs = dict(moves=torch.zeros(16, 2, dtype=torch.int32, device="cuda"),
                n_moves=torch.zeros(1, dtype=torch.int32, device="cuda"), status=B.new_status("cuda"))
    t1, c1, t2, c2, l2 = (torch.empty_like(x) for x in (t, c, t, c, l))
    s = torch.cuda.Stream()

    def step():
        B.resize_pages(t, l, new, c, P, block_table_out=t1, ref_count_out=c1, **bufs)
        B.copy_pages([cache], bufs["moves"], bufs["n_moves"], status=bufs["status"])
        B.fork_pages(t1, new, c1, par, P, block_table_out=t2, ref_count_out=c2, seq_lens_out=l2, **bufs)
        B.copy_pages([cache], bufs["moves"], bufs["n_moves"], status=bufs["status"])

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for add in (0, 5, 17):
        grown = np.minimum(lens + add, M * P).astype(np.int32)
        new.copy_(torch.from_numpy(grown))
        cache.random_(0, 256)
        host = cache.cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        a, ra, mv = OP.resize(table, lens, grown, ref, P)
        for src, dst in mv:
            host[dst] = host[src]
        want = OP.fork(a, grown, ra, par.cpu().numpy(), P)
        for src, dst in want[3]:
            host[dst] = host[src]
        assert int(bufs["status"].item()) == 0
        same(t2, want[0])
        same(c2, want[2])
        same(l2, want[1])
        same(cache, host)


def test_refusals(B):
    t = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    l = torch.zeros(2, dtype=torch.int32, device="cuda")
    c = torch.zeros(10, dtype=torch.int32, device="cuda")
    with pytest.raises(B.HpcError, match="own"):
        B.fork_pages(t, l, c, l, 16, block_table_out=t)
    with pytest.raises(B.HpcError, match="new_lens"):
        B.resize_pages(t, l, l[:1], c, 16)
    with pytest.raises(B.HpcError, match="page_size"):
        B.resize_pages(t, l, l, c, 0)
    with pytest.raises(B.HpcError, match="moves"):
        B.resize_pages(t, l, l, c, 16, moves=torch.zeros((1, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(B.HpcError, match="moves"):
        B.compact_pages(t, c, moves=torch.zeros((4, 2), dtype=torch.int32, device="cuda"))
    with pytest.raises(B.HpcError, match="ref_count_out"):
        B.compact_pages(t, c, ref_count_out=c[:5])
    with pytest.raises(B.HpcError, match="contiguous"):
        B.compact_pages(t[:, ::2], c)
    big = torch.zeros((8193, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(B.HpcError, match="8192"):
        B.resize_pages(big, big[:, 0].contiguous(), big[:, 0].contiguous(), c, 16)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    mv = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(B.HpcError, match="16"):
        B.copy_pages([torch.zeros((4, 24), dtype=torch.uint8, device="cuda")], mv, n)
    with pytest.raises(B.HpcError, match="one shape"):
        B.copy_pages([torch.zeros((4, 32), dtype=torch.uint8, device="cuda"),
                      torch.zeros((5, 32), dtype=torch.uint8, device="cuda")], mv, n)
    assert int(B.copy_pages([], mv, n).item()) == 0

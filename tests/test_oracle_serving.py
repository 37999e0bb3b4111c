"""Pins for oracle.pages, oracle.verify and oracle.prompt, and the host checks of the entry points they
belong to (argument errors return codes before any CUDA call)."""
import ctypes

import numpy as np
import pytest
import torch

from load_balanced_split_step_b200 import build
from oracle import pages as OP
from oracle import prompt as OQ
from oracle import verify as OV


@pytest.fixture(scope="module")
def B():
    build.build()
    from load_balanced_split_step_b200 import binding
    return binding


def test_pages_keep_the_counts_of_their_table():
    rng = np.random.default_rng(0)
    P, N, M = 4, 60, 6
    table, lens = np.full((6, M), -1), np.zeros(6, dtype=int)
    ref = np.zeros(N, dtype=int)
    for step in range(60):
        new = np.clip(lens + rng.integers(-6, 8, 6), 0, M * P)
        got = OP.resize(table, lens, new, ref, P)
        assert got is not None
        table, ref, moves = got
        old, lens = lens, new
        assert np.array_equal(ref, OP.counts(table, lens, N, P))
        assert all((row >= 0).sum() == OP.held(n, P) for row, n in zip(table, lens))
        grew = [row[OP.held(n, P) - 1] for row, n, o in zip(table, lens, old) if n > o and n % P]
        assert all(ref[p] == 1 for p in grew)  # a row writes to its own pages only
        got = OP.fork(table, lens, ref, rng.integers(-1, 6, 6), P)
        if got is None:
            continue
        table, lens, ref, moves = got
        assert np.array_equal(ref, OP.counts(table, lens, N, P))
        if step % 5 == 0:
            table, ref, page_map, moves = OP.compact(table, ref)
            n = int((ref > 0).sum())
            assert (ref[:n] > 0).all() and not ref[n:].any()
            assert np.array_equal(ref, OP.counts(table, lens, N, P))


def test_pages_hold_what_was_written():
    """Tokens written through the table are still there after forks, growth and compaction: a dict from
    (page, slot) to token stands for the cache."""
    rng = np.random.default_rng(1)
    P, N, M = 4, 64, 5
    cache = np.full((N, P), -1)
    table, lens, ref = np.full((4, M), -1), np.zeros(4, dtype=int), np.zeros(N, dtype=int)
    text = [[] for _ in range(4)]
    for step in range(80):
        new = np.clip(lens + rng.integers(-5, 6, 4), 0, M * P)
        table, ref, moves = OP.resize(table, lens, new, ref, P)
        for a, b in moves:
            cache[b] = cache[a]
        for r in range(4):
            text[r] = text[r][:new[r]]
            for pos in range(len(text[r]), new[r]):
                text[r].append(step * 100 + r * 10 + pos)
                cache[table[r, pos // P], pos % P] = text[r][-1]
        lens = new
        got = OP.fork(table, lens, ref, rng.integers(0, 4, 4), P)
        if step % 3 == 0 and got is not None:
            par = rng.integers(0, 4, 4)
            table, lens, ref, moves = OP.fork(table, lens, ref, par, P)
            text = [list(text[f]) for f in par]
            for a, b in moves:
                cache[b] = cache[a]
        if step % 7 == 0:
            table, ref, _, moves = OP.compact(table, ref)
            for a, b in moves:
                cache[b] = cache[a]
        for r in range(4):
            assert [int(cache[table[r, i // P], i % P]) for i in range(lens[r])] == text[r]


def test_verify_follows_the_target():
    """Exact for two tokens: P(first = 0) is the measure of the u that lead there, and equals p(0)."""
    p, q = np.array([[0.7, 0.3], [0.5, 0.5]]), np.array([[0.2, 0.8]])
    grid = (np.arange(200) + 0.5) / 200
    mass = 0.0
    for x, share in ((0, 0.2), (1, 0.8)):
        hits = [OV.verify_one([x], p, q, [a, 0.5], 1)[0][0] == 0 for a in grid]
        mass += share * np.mean(hits)  # the rest max(p - q, 0) is token 0 alone, whatever the last u
    assert abs(mass - 0.7) <= 0.005
    assert OV.sample(np.array([0.25, 0.0, 0.75]), 0.25) == 2 and OV.sample(np.array([0.25, 0.0, 0.75]), 0.0) == 0
    assert OV.sample(np.zeros(3), 0.5) == -1


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_attention_against_sdpa(causal):
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((7, 4, 8), (12, 2, 8), (12, 2, 8)))
    out, lse = OQ.attention(q, k, v, 0.3, causal)
    mask = torch.ones(7, 12, dtype=torch.bool).tril(5) if causal else torch.ones(7, 12, dtype=torch.bool)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.transpose(0, 1).repeat_interleave(2, 0), v.transpose(0, 1).repeat_interleave(2, 0),
        attn_mask=mask, scale=0.3).transpose(0, 1)
    assert np.abs(out - want.numpy()).max() < 1e-12
    s = torch.einsum("ihd,jhd->ihj", q, k.repeat_interleave(2, 1)) * 0.3
    s = s.masked_fill(~mask[:, None], -torch.inf)
    assert np.abs(lse - torch.logsumexp(s, -1).numpy()).max() < 1e-12
    out, lse = OQ.attention(q, k[:3], v[:3], 0.3, True)  # more queries than keys: the first see none
    assert not out[:4].any() and np.isinf(lse[:4]).all() and np.abs(out[4] - v[0].repeat_interleave(2, 0).numpy()).max() < 1e-12


def test_host_checks_of_the_page_calls(B):
    w, odd = ctypes.c_void_p(256), ctypes.c_void_p(260)
    lib = B._lib

    def resize(table=w, batch=2, pages=3, P=16, old=w, moves=w, cap=2, N=10):
        return lib.hpc_pages_resize(table, w, batch, pages, P, old, w, w, w, N, moves, cap, w, w, None)

    assert resize(table=None) == resize(old=None) == resize(moves=None) == B.HPC_ERR_ARG
    assert resize(batch=0) == resize(pages=0) == resize(P=0) == resize(N=0) == B.HPC_ERR_ARG
    assert resize(moves=odd) == B.HPC_ERR_ALIGN
    assert resize(batch=8193, cap=9000) == B.HPC_ERR_SHAPE
    assert resize(pages=1 << 20, P=1 << 12) == B.HPC_ERR_SHAPE
    assert resize(cap=1) == B.HPC_ERR_CAPACITY

    def fork(t_out=ctypes.c_void_p(512), l_out=ctypes.c_void_p(512), parents=w, rows=2, cap=2):
        return lib.hpc_pages_fork(w, w, 2, parents, t_out, l_out, rows, 3, 16, w, w, 10, w, cap, w, w, None)

    assert fork(parents=None) == B.HPC_ERR_ARG and fork(t_out=w) == B.HPC_ERR_ARG and fork(l_out=w) == B.HPC_ERR_ARG
    assert fork(rows=0) == B.HPC_ERR_ARG and fork(cap=1) == B.HPC_ERR_CAPACITY
    assert lib.hpc_pages_compact(w, w, 2, 3, w, w, 10, None, w, 5, w, w, None) == B.HPC_ERR_ARG
    assert lib.hpc_pages_compact(w, w, 2, 3, w, w, 10, w, w, 4, w, w, None) == B.HPC_ERR_CAPACITY
    assert resize(batch=4096, pages=1 << 20, P=1, cap=4096) == B.HPC_ERR_SHAPE
    assert lib.hpc_pages_fork(w, w, 4096, w, ctypes.c_void_p(512), ctypes.c_void_p(512), 2, 1 << 20, 1, w, w, 10, w, 2, w, w,
                              None) == B.HPC_ERR_SHAPE
    ptrs = (ctypes.c_void_p * 2)(256, 264)
    assert lib.hpc_pages_copy(None, 1, 16, 4, w, 1, w, w, None) == B.HPC_ERR_ARG
    assert lib.hpc_pages_copy(ptrs, 1, 24, 4, w, 1, w, w, None) == B.HPC_ERR_SHAPE
    assert lib.hpc_pages_copy(ptrs, 2, 32, 4, w, 1, w, w, None) == B.HPC_ERR_ALIGN
    assert lib.hpc_pages_copy(ptrs, 1, 32, 4, w, 0, w, w, None) == B.HPC_OK  # nothing to do


def test_host_checks_of_verify_and_prologue(B):
    w = ctypes.c_void_p(256)
    lib = B._lib

    def verify(drafts=w, p=w, ps=100, q=w, qs=100, dt=B.HPC_FP32, seq=w, batch=2, T=3, V=100, new=w):
        return lib.hpc_verify_drafts(drafts, p, ps, q, qs, dt, w, None, seq, batch, T, V, w, w, new, w, None)

    assert verify(p=None) == verify(drafts=None) == verify(seq=None) == B.HPC_ERR_ARG
    assert verify(ps=99) == verify(qs=99) == verify(batch=0) == verify(V=0) == verify(T=-1) == B.HPC_ERR_ARG
    assert verify(dt=B.HPC_E4M3) == B.HPC_ERR_DTYPE and verify(T=257) == B.HPC_ERR_SHAPE

    def pro(tokens=4, qkv=w, cu=w, kv=B.HPC_BF16, ks=None, D=64, heads=8, theta=1e6, q_out=w):
        return lib.hpc_prompt_prologue(qkv, tokens, cu, 2, w, w, 1e-6, theta, q_out, None, w, w, kv, 0, ks, ks, 4, 16, w,
                                       3, w, heads, 2, D, w, None)

    assert pro(qkv=None) == pro(cu=None) == pro(tokens=-1) == pro(theta=0.0) == pro(kv=B.HPC_E4M3) == B.HPC_ERR_ARG
    assert pro(kv=B.HPC_FP32) == B.HPC_ERR_DTYPE and pro(D=96) == pro(heads=7) == pro(tokens=1 << 31) == B.HPC_ERR_SHAPE
    assert pro(q_out=ctypes.c_void_p(264)) == B.HPC_ERR_ALIGN and pro(tokens=0) == B.HPC_OK


def test_host_checks_of_prompt_attention(B):
    w, odd = ctypes.c_void_p(256), ctypes.c_void_p(264)
    lib = B._lib

    def packed(q=w, k=w, v=w, stride=1024, kstride=256, tokens=4, kv=4, cu=w, cu_k=None, batch=2, H=8, Hkv=2, D=128,
               scale=0.1, out=w, work=w, part=None, room=0):
        return lib.hpc_prompt_attention(q, stride, D, k, kstride, D, v, kstride, D, tokens, kv, cu, cu_k, batch, H, Hkv, D, 1,
                                        scale, out, None, work, part, room, w, None)

    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(out=None), dict(work=None), dict(room=64),
                dict(tokens=-1), dict(kv=-1, cu_k=w), dict(kv=5), dict(batch=0), dict(H=0), dict(Hkv=0), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(tokens=1 << 31)):
        assert packed(**bad) == B.HPC_ERR_ARG, bad
    for bad in (dict(H=7), dict(H=6), dict(H=32), dict(D=96), dict(D=256)):
        assert packed(**bad) == B.HPC_ERR_SHAPE, bad
    for bad in (dict(q=odd), dict(out=odd), dict(part=odd, room=64), dict(stride=1028)):
        assert packed(**bad) == B.HPC_ERR_ALIGN, bad
    assert packed(tokens=0, kv=0, q=None, out=None, k=None, v=None) == B.HPC_OK  # nothing to do

    def paged(k=w, kv=B.HPC_BF16, lay=B.HPC_HND, N=4, P=16, table=w, M=3, lens=w, tokens=0):
        return lib.hpc_prompt_attention_paged(w, 1024, 128, k, w, kv, lay, N, P, table, M, lens, tokens, w, 2, 8, 2, 128, 0.1,
                                              w, None, w, None, 0, w, None)

    assert paged(k=None) == paged(table=None) == paged(lens=None) == paged(lay=2) == paged(N=0) == paged(M=0) == B.HPC_ERR_ARG
    assert paged(kv=B.HPC_E4M3) == B.HPC_ERR_DTYPE
    assert paged(P=8) == paged(P=48) == paged(P=256) == paged(M=1 << 28) == B.HPC_ERR_SHAPE
    assert paged(k=odd) == B.HPC_ERR_ALIGN and paged() == B.HPC_OK
    assert lib.hpc_prompt_attention_partial_bytes(96) == 0 and lib.hpc_prompt_attention_partial_bytes(64) > 0


def test_host_checks_of_gather_tokens(B):
    w, odd = ctypes.c_void_p(256), ctypes.c_void_p(264)
    lib = B._lib

    def gather(k=w, kv=B.HPC_BF16, lay=B.HPC_HND, ks=None, N=4, P=16, table=w, M=3, lens=w, batch=2, H=2, D=128, n=8, ko=w,
               cu=w):
        return lib.hpc_gather_tokens(k, w, kv, lay, ks, ks, N, P, table, M, lens, batch, H, D, n, ko, w, cu, w, None)

    for bad in (dict(k=None), dict(table=None), dict(lens=None), dict(cu=None), dict(ko=None), dict(lay=2), dict(N=0),
                dict(P=0), dict(M=0), dict(batch=0), dict(H=0), dict(n=-1), dict(n=1 << 31), dict(kv=B.HPC_E4M3)):
        assert gather(**bad) == B.HPC_ERR_ARG, bad
    assert gather(kv=B.HPC_FP32) == B.HPC_ERR_DTYPE
    assert gather(D=96) == gather(batch=8193) == gather(H=65537) == B.HPC_ERR_SHAPE
    assert gather(k=odd) == gather(ko=odd) == B.HPC_ERR_ALIGN

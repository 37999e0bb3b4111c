"""Prompt attention over cached tokens by way of packed rows: what it answers to lengths that do not hold together."""
import ctypes
import math

import pytest
import torch

from tests.test_gpu_gather_tokens import cache
from tests.test_gpu_prompt_attention import cu, draw


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def test_host_checks(B):
    w = ctypes.c_void_p(256)

    def gather(k=w, cq=w, D=128, kv=B.HPC_BF16):
        return B._lib.hpc_gather_prompt_tokens(k, w, kv, B.HPC_HND, None, None, 4, 16, w, 3, w, cq, 2, 2, D, 8, w, w, w, w, None)

    assert gather(cq=None) == gather(k=None) == gather(kv=B.HPC_E4M3) == B.HPC_ERR_ARG
    assert gather(D=96) == B.HPC_ERR_SHAPE and gather(kv=B.HPC_FP32) == B.HPC_ERR_DTYPE


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("short", [39, 1, 0, -1, 10 ** 6])
def test_fewer_cached_tokens_than_queries(B, kv, short):
    """The second of three requests brings 40 queries and says that fewer tokens (or an impossible number) are cached: the
    call says so, by either way in, that request gets zeros and -inf, and the others get what they get alone."""
    lens, total, Hq, Hkv, D, P = (30, 40, 7), (200, 40, 90), 4, 2, 64, 16
    (kp, vp), table, seq, _, kw = cache(1, total, Hkv, D, P, "HND", kv)
    q, c = draw(3, sum(lens), Hq, D), cu(lens)
    want, want_lse, st = B.prompt_attention_paged(q, kp, vp, table, seq, c, kv_tokens=330, return_lse=True, **kw)
    assert int(st.item()) == 0
    seq[1] = short
    out, lse, st = B.prompt_attention_paged(q, kp, vp, table, seq, c, kv_tokens=330, return_lse=True, **kw)
    assert int(st.item()) == B.DEV_STATUS["bad_seqlen"]
    for a, b in ((0, 30), (70, 77)):
        assert torch.equal(out[a:b], want[a:b]) and torch.equal(lse[a:b], want_lse[a:b])
    assert not out[30:70].any() and (lse[30:70] == -math.inf).all()
    if kv == "bf16":
        assert int(B.prompt_attention_paged(q, kp, vp, table, seq, c)[2].item()) == B.DEV_STATUS["bad_seqlen"]
    # without queries to count, a short request is as good as any
    if 0 <= short < 40:
        _, _, boundaries, st = B.gather_tokens(kp, vp, table, seq, 330, **kw)
        assert int(st.item()) == 0 and boundaries.tolist() == cu((200, short, 90)).tolist()


@pytest.mark.gpu
def test_refusals(B):
    (kp, vp), table, seq, _, kw = cache(1, (5, 9), 2, 64, 16, "HND", "bf16")
    for cq, what in ((cu([5]), "cu_seqlens"), (cu([5, 9]).long(), "cu_seqlens"), (cu([5, 9]).cpu(), "cu_seqlens")):
        with pytest.raises(B.HpcError, match=what):
            B.gather_tokens(kp, vp, table, seq, 14, cu_queries=cq, **kw)

"""Prompt attention over cached tokens by way of packed rows: what it answers to lengths that do not hold together, and how
far an E4M3 cache's values are from those that its codes and scales stand for.

Tolerance of the latter. A row's value is code x scale rounded to bf16: off by 2^-8 and 2^-23 (the product in fp32) relative, K
and V alike. That moves a score by at most S = (2^-8 + 2^-23) sm_scale max_j sum_d |q_d k_jd|, and the sums of the kernel by E
(as in test_gpu_prompt_attention), so that a normalised weight changes by a factor within exp(+-2 (S + E)); it is rounded to
bf16 too. With A = sum_j p_j |v_j|: |err| <= A (exp(2 (S + E)) (1 + 2^-8 + 2^-20)^2 - 1), and half a bf16 step of the
result."""
import ctypes
import math

import pytest
import torch

from tests.test_gpu_gather_tokens import cache
from tests.test_gpu_prompt_attention import cu, draw, reference


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
@pytest.mark.parametrize("layout,D", [("NHD", 128), ("HND", 64)])
def test_against_the_values_of_the_cache(B, layout, D):
    lens, total, Hq, Hkv, P = (1, 130, 7, 300), (1, 130, 1007, 2300), 8, 2, 16
    (kp, vp), table, seq, _, _ = cache(P, total, Hkv, D, P, layout, "bf16")
    scale = torch.tensor([0.021, 0.0537], device="cuda")
    shape = (-1, 1, 1) if layout == "HND" else (-1, 1)
    kp, vp = [(x.float() / scale.view(shape)).to(torch.float8_e4m3fn) for x in (kp, vp)]
    q = draw(3, sum(lens), Hq, D)
    out, lse, st = B.prompt_attention_paged(q, kp, vp, table, seq, cu(lens), return_lse=True, kv_tokens=sum(total),
                                            kv_dtype="e4m3", kv_layout=layout, k_scale=scale, v_scale=scale)
    assert int(st.item()) == 0
    k, v = [x.double() * scale.double().view(shape) for x in (kp, vp)]  # what the codes stand for
    if layout == "HND":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    o = 0
    for r, (n, m) in enumerate(zip(lens, total)):
        pages = table[r, :-(-m // P)].long()
        want, ls, A, E = reference(q[o:o + n], k[pages].flatten(0, 1)[:m], v[pages].flatten(0, 1)[:m], D ** -0.5, True)
        moved = E / (D * 2.0 ** -24) * (2.0 ** -8 + 2.0 ** -23) + E
        tol = A * (torch.exp(2 * moved)[..., None] * (1 + 2.0 ** -8 + 2.0 ** -20) ** 2 - 1)
        tol = tol + (want.abs() + tol) * 2.0 ** -8
        err = (out[o:o + n].double() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        assert bool(((lse[o:o + n].double() - ls).abs() <= moved + 2.0 ** -20 * (1 + ls.abs())).all())
        o += n


@pytest.mark.gpu
def test_refusals(B):
    (kp, vp), table, seq, _, kw = cache(1, (5, 9), 2, 64, 16, "HND", "bf16")
    for cq, what in ((cu([5]), "cu_seqlens"), (cu([5, 9]).long(), "cu_seqlens"), (cu([5, 9]).cpu(), "cu_seqlens")):
        with pytest.raises(B.HpcError, match=what):
            B.gather_tokens(kp, vp, table, seq, 14, cu_queries=cq, **kw)

"""Verification of drafted tokens against the fp64 oracle. Tokens and counts are whole numbers, so every
comparison is for equality. Sums of up to 2^17 probabilities in fp64 differ by order by about 1e-11 of the
total at most, and no test's random number lies that close to a border of the cumulative sum except
where the sums are exact (dyadic probabilities)."""
import numpy as np
import pytest
import torch

from oracle import verify as OV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def case(seed, Bn, T, V, dtype, onehot=False, peak=3.0, agree=0.7):
    g = torch.Generator().manual_seed(seed)
    logits = peak * torch.randn((Bn, T + 1, V), generator=g)
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits[:, :T] + agree * torch.randn((Bn, T, V), generator=g), -1)
    x = torch.zeros((Bn, T), dtype=torch.int32)
    if T:
        x = torch.multinomial(q.reshape(Bn * T, V), 1, generator=g).reshape(Bn, T).to(torch.int32)
    u = torch.rand((Bn, T + 1), generator=g)
    n = torch.randint(0, T + 1, (Bn,), generator=g, dtype=torch.int32)
    lens = torch.randint(T + 1, 1000, (Bn,), generator=g, dtype=torch.int32)
    return x, p.to(dtype), None if onehot else q.to(dtype), u, n, lens


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check(B, x, p, q, u, n=None, lens=None, status=0):
    xd, pd, qd, ud, nd, ld = cuda(x, p, q, u, n, lens)
    tokens, acc, new, st = B.verify_drafts(xd, pd, qd, ud, draft_lens=nd, seq_lens=ld)
    assert int(st.item()) == status
    Bn, T = x.shape
    for r in range(Bn):
        k = T if n is None else min(max(int(n[r]), 0), T)
        want, a = OV.verify_one(x[r].tolist(), p[r].double().numpy(), None if q is None else q[r].double().numpy(),
                                u[r].tolist(), k)
        assert tokens[r].tolist() == want.tolist(), r
        assert int(acc[r]) == a, r
        if lens is not None:
            assert int(new[r]) == int(lens[r]) - k + a, r
    return tokens, acc


@pytest.mark.parametrize("V", [1, 2, 31, 257, 4096, 32000, 131071])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("onehot", [False, True])
def test_against_the_oracle(B, V, dtype, onehot):
    Bn, T = (3, 3) if V > 5000 else (17, 5)
    x, p, q, u, n, lens = case(V, Bn, T, V, dtype, onehot)
    check(B, x, p, q, u, n, lens)
    check(B, x, p, q, u)


@pytest.mark.parametrize("T", [0, 1, 7, 64, 256])
def test_draft_counts(B, T):
    x, p, q, u, n, lens = case(T, 2, T, 50, torch.float32, agree=0.05)
    check(B, x, p, q, u, None, lens)
    check(B, x, p, q, u, n, lens)


def test_borders(B):
    """Dyadic probabilities: every product and sum is exact, so the borders themselves are tested.
    A draft is kept for u q < p only; the draw takes the lowest entry whose sum passes u."""
    V = 1024
    p = torch.full((6, 2, V), 1.0 / V)
    q = torch.full((6, 1, V), 1.0 / V)
    q[:, 0, 7] = 4.0 / V
    x = torch.full((6, 1), 7, dtype=torch.int32)
    # u q < p: u < 1/4. At u = 1/4 the draft is rejected.
    u = torch.tensor([[0.25, 0.0], [0.25 - 2.0 ** -20, 0.5], [0.0, 0.5 - 2.0 ** -20], [0.1, 0.0], [0.1, 1 - 2.0 ** -24],
                      [0.2, 511.0 / 1024]])
    p[0, 0, 900] = 2.0 / V  # the rest max(p - q, 0) of row 0 is this entry alone
    tokens, acc = check(B, x, p, q, u)
    assert acc.tolist() == [0, 1, 1, 1, 1, 1]
    assert tokens[:, 0].tolist() == [900, 7, 7, 7, 7, 7]
    assert tokens[:, 1].tolist() == [-1, 512, 511, 0, 1023, 511]


def test_rest_without_mass_takes_the_target(B):
    V = 300
    p = torch.zeros((3, 2, V))
    p[:, :, 5], p[:, :, 290] = 0.25, 0.75
    q = p[:, :1].clone()
    x = torch.tensor([[4], [5], [290]], dtype=torch.int32)  # 4 has no mass in either
    u = torch.tensor([[0.0, 0.5], [1.0, 0.1], [1.0, 0.25]])  # u = 1 rejects a certain match
    tokens, acc = check(B, x, p, q, u)
    assert acc.tolist() == [0, 0, 0] and tokens[:, 0].tolist() == [290, 5, 290]
    one = torch.zeros((1, 2, V))
    one[:, :, 9] = 1.0  # a one-hot draft of the target's only token, rejected by u = 1
    tokens, _ = check(B, torch.tensor([[9]], dtype=torch.int32), one, None, torch.tensor([[1.0, 0.3]]))
    assert tokens[0].tolist() == [9, -1]


@pytest.mark.parametrize("V", [999, 40001, 131072])
@pytest.mark.parametrize("bads", [("nan", "inf", -1.0, "-inf"), ("nan", -1.0)])
def test_values_that_are_no_probabilities_count_as_zero(B, V, bads):
    x, p, q, u, n, lens = case(77, 4, 2, V, torch.float32)
    for bad, at in zip(bads, (3, V // 2, V - 1, 0)):
        p[:, :, at] = float(bad)
        q[:, :, (at + 1) % V] = float(bad)
    check(B, x, p, q, u, n, lens)
    u[:, -1] = float("nan")  # no sum passes a NaN: the last entry with mass
    check(B, x, p, q, u, n, lens)
    u[:, -1] = 1.5
    check(B, x, p, q, u, n, lens)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [700, 40001, 131071])
def test_an_infinity_of_the_draft_counts_as_zero(B, V, dtype):
    # Half of the target's mass lies where the draft's value is infinite: the rest there is the target's share.
    p, q = torch.full((4, 2, V), 2.0**-20, dtype=dtype), torch.full((4, 1, V), 2.0**-19, dtype=dtype)
    for r, at in enumerate((V // 2, V // 3, 5, V - 1)):
        p[r, 0, at], q[r, 0, at], p[r, 0, V // 5] = 0.5, float("inf"), 0.25
    q[:, 0, V // 5] = 2.0**-21  # exact sums: 0.25 - 2^-21 and 0.5 are all that is left
    x = torch.full((4, 1), V // 7, dtype=torch.int32)
    for draw in (0.125, 0.375, 0.75):
        check(B, x, p, q, torch.tensor([[0.9, draw]] * 4))


def test_status_bits(B):
    x, p, q, u, n, _ = case(5, 4, 3, 64, torch.float32, agree=0.0)
    u[:] = 0.0
    bad = x.clone()
    bad[1, 1], bad[2, 0] = 64, -1
    _, acc = check(B, bad, p, q, u, status=B.DEV_STATUS["bad_index"])
    assert acc.tolist() == [3, 1, 0, 3]
    check(B, bad, p, None, u, status=B.DEV_STATUS["bad_index"])
    n = torch.tensor([-3, 4, 1, 0], dtype=torch.int32)
    check(B, x, p, q, u, n, status=B.DEV_STATUS["bad_seqlen"])
    p[3] = 0.0
    tokens, acc = check(B, x, p, q, u, status=B.DEV_STATUS["bad_probs"])
    assert int(acc[3]) == 0 and tokens[3].tolist() == [-1, -1, -1, -1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padded_rows_and_offsets(B, dtype):
    """A vocabulary padded to a wider row, and tensors that start at odd elements."""
    x, p, q, u, n, lens = case(9, 3, 4, 1001, dtype)
    wide_p = torch.full((3 * 5 * 1030 + 3,), float("nan"), dtype=dtype, device="cuda")
    wide_q = torch.full((3 * 4 * 1017 + 1,), float("nan"), dtype=dtype, device="cuda")
    pv = wide_p[3:].view(3, 5, 1030)[:, :, :1001]
    qv = wide_q[1:].view(3, 4, 1017)[:, :, :1001]
    pv.copy_(p)
    qv.copy_(q)
    a = B.verify_drafts(*cuda(x), pv, qv, *cuda(u), draft_lens=n.cuda())
    b = B.verify_drafts(*cuda(x, p, q, u), draft_lens=n.cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(B, x, p, q, u, n)


def test_distribution_is_the_targets(B):
    """Over many random numbers the first emitted token follows p, whatever the draft: counts against a
    chi-square bound (V - 1 = 15 degrees of freedom; 50 has a tail of about 1e-5), seed fixed."""
    V, Bn = 16, 40000
    g = torch.Generator().manual_seed(1)
    p = torch.softmax(torch.randn(V, generator=g), -1)
    q = torch.softmax(torch.randn(V, generator=g), -1)
    x = torch.multinomial(q, Bn, replacement=True, generator=g).to(torch.int32)[:, None]
    u = torch.rand((Bn, 2), generator=g)
    tokens, _, _, _ = B.verify_drafts(*cuda(x, p.expand(Bn, 2, V).contiguous(), q.expand(Bn, 1, V).contiguous(), u))
    count = torch.bincount(tokens[:, 0].long(), minlength=V).cpu().double()
    want = p.double() / p.double().sum() * Bn
    assert float(((count - want) ** 2 / want).sum()) < 50


def test_two_streams_and_a_graph(B):
    x, p, q, u, n, lens = cuda(*case(31, 5, 3, 5000, torch.float32))
    want = B.verify_drafts(x, p, q, u, draft_lens=n, seq_lens=lens)
    torch.cuda.synchronize()
    outs = [torch.empty_like(want[0]) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, o in zip(streams, outs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                B.verify_drafts(x, p, q, u, draft_lens=n, out_tokens=o)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    acc, st = torch.empty_like(want[1]), B.new_status("cuda")
    with torch.cuda.graph(g):
        B.verify_drafts(x, p, q, u, draft_lens=n, out_tokens=outs[2], accepted=acc, status=st)
    u2 = torch.rand_like(u)
    u.copy_(u2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[0])
    again = B.verify_drafts(x, p, q, u2, draft_lens=n)
    assert torch.equal(outs[2], again[0]) and torch.equal(acc, again[1])


def test_refusals(B):
    x, p, q, u, n, lens = cuda(*case(2, 2, 3, 40, torch.float32))
    for args, kw, what in (((x, p.half(), q, u), {}, "dtype"), ((x, p, q.bfloat16(), u), {}, "draft_probs"),
                           ((x, p[:, :3], q, u), {}, "target_probs"), ((x, p, q, u[:, :3]), {}, "uniforms"),
                           ((x.long(), p, q, u), {}, "draft_tokens"), ((x, p, q, u), dict(draft_lens=n[:1]), "draft_lens"),
                           ((x, p[:, :, ::2], q[:, :, ::2], u), {}, "contiguous"),
                           ((x, p.transpose(0, 1).contiguous().transpose(0, 1), q, u), {}, "rows"),
                           ((x, p, q, u), dict(new_lens=n), "seq_lens"),
                           ((x, p.cpu(), q, u), {}, "CUDA")):
        with pytest.raises(B.HpcError, match=what):
            B.verify_drafts(*args, **kw)
    many = torch.zeros((1, 257), dtype=torch.int32, device="cuda")
    with pytest.raises(B.HpcError, match="256"):
        B.verify_drafts(many, torch.ones((1, 258, 4), device="cuda"), None, torch.zeros((1, 258), device="cuda"))

"""Prompt attention (packed and paged) against softmax(q k^T) v in 64 bits.

Tolerances, per element. The weights are rounded to bf16 for the product with V (at most half a step,
2^-8 relative, each) and so is the result: |err| <= 2^-8 A + 2^-8 |o| (1 + 2^-8), with A = sum_j p_j |v_j| over
the normalised weights. The scores are fp32 sums of D products, whose error is at most
E = D 2^-24 sm_scale max_j sum_d |q_d k_jd|; with the exponential's 2^-22 that changes every weight by
at most about 2 E + 2^-20 relative, and the log-sum-exp by E + 2^-20 (1 + |lse|)."""
import math

import numpy as np
import pytest
import torch

from oracle import prompt as OR

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def reference(q, k, v, scale, causal):
    """One sequence in fp64 on the device: (out, lse, A, E); query i is at key position i + m - n."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    q, k, v = q.double(), k.double(), v.double()
    out, lse = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device), torch.full(
        (n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    A, E = torch.zeros_like(out), torch.zeros_like(lse)
    if m == 0:
        return out, lse, A, E
    seen = torch.ones(n, m, dtype=torch.bool, device=q.device)
    if causal:
        seen = seen.tril(m - n)
    some = seen.any(1)
    for h in range(Hq):
        g = h * Hkv // Hq
        s = (q[:, h] @ k[:, g].T * scale).masked_fill(~seen, -math.inf)
        ls = torch.logsumexp(s, 1)
        p = torch.where(some[:, None], torch.exp(s - ls[:, None]), torch.zeros_like(s))
        out[:, h], A[:, h] = p @ v[:, g], p @ v[:, g].abs()
        lse[:, h] = ls
        E[:, h] = D * 2.0 ** -24 * scale * (q[:, h].abs() @ k[:, g].abs().T).amax(1)
    return out, lse, A, E


def check(got, lse, want):
    o, ls, A, E = want
    tol = A * (2.0 ** -8 + 2.0 * E[..., None] + 2.0 ** -20) + o.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + 1e-37
    err = (got.double() - o).abs()
    assert bool((err <= tol).all()), f"max error / tolerance {float((err / tol).max())}"
    if lse is not None:
        seen = ls > -math.inf
        assert torch.equal(lse > -math.inf, seen)
        d = (lse.double() - ls).abs()
        assert bool((d[seen] <= (E + 2.0 ** -20 * (1 + ls.abs()))[seen]).all())


def cu(lens, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + start, dtype=torch.int32, device="cuda")


def draw(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


@pytest.mark.parametrize("lens", [(1,), (2, 1, 3), (15, 16, 17), (127, 128, 129, 1), (255, 0, 256, 257, 0), (700, 5, 33),
                                  (1000,), (1,) * 70 + (40,) * 7])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 2, 64), (8, 1, 128), (4, 4, 128), (6, 3, 128)])
def test_packed_causal(B, lens, Hq, Hkv, D):
    n = sum(lens)
    qkv = draw(n + Hq, n, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out, lse, st = B.prompt_attention(q, k, v, cu(lens), return_lse=True)
    assert int(st.item()) == 0
    o = 0
    for x in lens:
        if x:
            check(out[o:o + x], lse[o:o + x], reference(q[o:o + x], k[o:o + x], v[o:o + x], D ** -0.5, True))
        o += x


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,keys", [((5, 1, 130), (9, 700, 130)), ((40, 3, 0, 7), (17, 3, 5, 0)), ((300,), (1025,)),
                                       ((64, 64), (128, 64)), ((513,), (100,))])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (2, 2, 64), (4, 1, 64)])
def test_keys_of_another_length(B, causal, lens, keys, Hq, Hkv, D):
    """More keys than queries, fewer (rows that see none), and none at all."""
    q, k, v = draw(1, sum(lens), Hq, D), draw(2, sum(keys), Hkv, D), draw(3, sum(keys), Hkv, D)
    out, lse, st = B.prompt_attention(q, k, v, cu(lens), cu_seqlens_k=cu(keys), causal=causal, return_lse=True, sm_scale=0.2)
    assert int(st.item()) == 0
    o = p = 0
    for x, y in zip(lens, keys):
        if x:
            check(out[o:o + x], lse[o:o + x], reference(q[o:o + x], k[p:p + y], v[p:p + y], 0.2, causal))
        o, p = o + x, p + y


@pytest.mark.parametrize("lens", [(4096, 17, 2050), (9000,)])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 128), (4, 4, 64)])
def test_long(B, lens, Hq, Hkv, D):
    n = sum(lens)
    q, k, v = draw(5, n, Hq, D, scale=2.0), draw(6, n, Hkv, D, scale=2.0), draw(7, n, Hkv, D)
    out, lse, st = B.prompt_attention(q, k, v, cu(lens), return_lse=True)
    assert int(st.item()) == 0
    o = 0
    for x in lens:
        check(out[o:o + x], lse[o:o + x], reference(q[o:o + x], k[o:o + x], v[o:o + x], D ** -0.5, True))
        o += x


@pytest.mark.parametrize("lens,keys", [((1,), (9000,)), ((16,), (30011,)), ((300, 2, 5), (20000, 700, 1537)),
                                       ((40, 40, 33, 1), (5000, 129, 0, 12000)), ((1700,), (1700,)), ((2500, 3), (2500, 6001)),
                                       ((7,) * 9, (3000,) * 9)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (2, 2, 64), (16, 2, 128), (1, 1, 64)])
def test_cut_along_the_keys(B, lens, keys, Hq, Hkv, D):
    """Few queries on many keys: units are cut into parts that are joined, the same way every time."""
    q, k, v = draw(1, sum(lens), Hq, D, scale=2.0), draw(2, sum(keys), Hkv, D), draw(3, sum(keys), Hkv, D)
    for causal in (True, False):
        out, lse, st = B.prompt_attention(q, k, v, cu(lens), cu_seqlens_k=cu(keys), causal=causal, return_lse=True)
        assert int(st.item()) == 0
        o = p = 0
        for x, y in zip(lens, keys):
            check(out[o:o + x], lse[o:o + x], reference(q[o:o + x], k[p:p + y], v[p:p + y], D ** -0.5, causal))
            o, p = o + x, p + y
        for _ in range(3):
            again = B.prompt_attention(q, k, v, cu(lens), cu_seqlens_k=cu(keys), causal=causal, return_lse=True)
            assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("room", [0, 1, 9, 10 ** 9])
def test_any_room_for_parts_will_do(B, room):
    """Through the C call: scratch for no part, for one, for a few, for all."""
    lens, keys, Hq, Hkv, D = (40, 9), (7000, 4000), 4, 2, 64
    q, k, v = draw(1, 49, Hq, D), draw(2, 11000, Hkv, D), draw(3, 11000, Hkv, D)
    full = B._lib.hpc_prompt_attention_partial_bytes(D)
    slot = 2 * 128 * (D + 2) * 4
    nbytes = min(16384 + room * slot, full)  # the list of cut units, then the parts
    partial = torch.full((nbytes + 256,), 255, dtype=torch.uint8, device="cuda")
    work = torch.zeros(B.PROMPT_WORK_WORDS, dtype=torch.int32, device="cuda")
    out, lse, st = torch.empty_like(q), torch.empty(49, Hq, device="cuda"), B.new_status("cuda")
    cq, ck = cu(lens), cu(keys)
    B._launch("hpc_prompt_attention", q.device, q.data_ptr(), Hq * D, D, k.data_ptr(), Hkv * D, D, v.data_ptr(), Hkv * D, D,
              49, 11000, cq.data_ptr(), ck.data_ptr(), 2, Hq, Hkv, D, 1, 0.125, out.data_ptr(), lse.data_ptr(),
              work.data_ptr(), partial.data_ptr(), nbytes, st.data_ptr())
    assert int(st.item()) == 0 and (partial[nbytes:] == 255).all()
    o = p = 0
    for x, y in zip(lens, keys):
        check(out[o:o + x], lse[o:o + x], reference(q[o:o + x], k[p:p + y], v[p:p + y], 0.125, True))
        o, p = o + x, p + y


@pytest.mark.parametrize("which,at", [("v", 8990), ("v", 100), ("k", 5000)])
def test_cut_with_values_that_are_not_finite(B, which, at):
    q, k, v = draw(1, 30, 8, 128), draw(2, 9000, 1, 128), draw(3, 9000, 1, 128)
    x = {"k": k.clone(), "v": v.clone()}
    x[which][at, 0, 7] = math.nan
    out, lse, st = B.prompt_attention(q, x["k"], x["v"], cu([30]), cu_seqlens_k=cu([9000]), return_lse=True)
    assert int(st.item()) == 0
    before = max(0, at - 8970)  # queries that do not see it
    want = reference(q, k, v, 128 ** -0.5, True)
    check(out[:before], lse[:before], [w[:before] for w in want])
    seen = out[before:]
    if which == "v":
        assert torch.isnan(seen[:, :, 7]).all() and not torch.isnan(seen[:, :, :7]).any()
        check(out[:, :, 8:], lse, [want[0][:, :, 8:], want[1], want[2][:, :, 8:], want[3]])
    else:
        assert torch.isnan(seen).all() and torch.isnan(lse[before:]).all()


@pytest.mark.parametrize("P,layout", [(16, "HND"), (64, "NHD"), (128, "HND")])
def test_cut_paged(B, P, layout):
    lens, ctx = (3, 64, 1), (20000, 5000, 2047)
    kp, vp, table, seq, ks, vs = paged(P, lens, ctx, 2, 128, P, layout)
    q = draw(3, sum(lens), 8, 128)
    out, lse, st = B.prompt_attention_paged(q, kp, vp, table, seq, cu(lens), kv_layout=layout, return_lse=True)
    assert int(st.item()) == 0
    o = 0
    for r, x in enumerate(lens):
        check(out[o:o + x], lse[o:o + x], reference(q[o:o + x], ks[r], vs[r], 128 ** -0.5, True))
        o += x


def test_reference_is_the_oracle():
    q, k, v = draw(1, 9, 4, 64), draw(2, 20, 2, 64), draw(3, 20, 2, 64)
    for causal in (True, False):
        o, ls, _, _ = reference(q, k, v, 0.3, causal)
        want, wls = OR.attention(q, k, v, 0.3, causal)
        assert np.abs(o.cpu().numpy() - want).max() < 1e-12 and np.abs(ls.cpu().numpy() - wls).max() < 1e-12


@pytest.mark.parametrize("kind", ["growing", "shrinking", "huge", "equal", "spread"])
def test_scores_of_every_size(B, kind):
    """The running reference: scores that grow block by block (every block rescales), one far above the
    rest, equal ones, and rows whose first keys are far below the later ones."""
    n, Hq, Hkv, D = 900, 8, 2, 128
    q, k, v = draw(11, n, Hq, D), draw(12, n, Hkv, D), draw(13, n, Hkv, D)
    pos = torch.arange(n, device="cuda", dtype=torch.float32)[:, None]
    if kind in ("growing", "shrinking"):
        q[..., 0] = 4.0
        k[..., 0] = (pos if kind == "growing" else n - pos) * 0.5
    elif kind == "huge":
        k[400] = k[400] * 200
        k[50] = k[50] * 1000
    elif kind == "equal":
        q[:] = 0
    else:
        q[..., 1] = 30.0
        k[..., 1] = torch.where(pos < 300, -50.0, 10.0) * (1 + 0.001 * pos)
    out, lse, st = B.prompt_attention(q, k, v, cu([n]), return_lse=True)
    assert int(st.item()) == 0
    check(out, lse, reference(q, k, v, D ** -0.5, True))


def paged(seed, lens, ctx, Hkv, D, P, layout):
    """Pages in random order; unused slots and pages hold NaN."""
    g = torch.Generator().manual_seed(seed)
    total = [a + b for a, b in zip(lens, ctx)]
    need = [-(-t // P) for t in total]
    N = sum(need) + 3
    shape = (N, P, Hkv, D)
    kp, vp = torch.full(shape, math.nan, dtype=torch.bfloat16), torch.full(shape, math.nan, dtype=torch.bfloat16)
    perm = torch.randperm(N, generator=g)
    table = torch.full((len(lens), max(need) + 2), -1, dtype=torch.int32)
    o, ks, vs = 0, [], []
    for r, t in enumerate(total):
        k, v = (torch.randn((t, Hkv, D), generator=g).to(torch.bfloat16) for _ in range(2))
        ids = perm[o:o + need[r]]
        o += need[r]
        table[r, :need[r]] = ids
        for j in range(need[r]):
            e = min(P, t - j * P)
            kp[ids[j], :e], vp[ids[j], :e] = k[j * P:j * P + e], v[j * P:j * P + e]
        ks.append(k.cuda())
        vs.append(v.cuda())
    if layout == "HND":
        kp, vp = kp.transpose(1, 2).contiguous(), vp.transpose(1, 2).contiguous()
    return kp.cuda(), vp.cuda(), table.cuda(), torch.tensor(total, dtype=torch.int32, device="cuda"), ks, vs


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (4, 2, 64)])
def test_paged(B, P, layout, Hq, Hkv, D):
    lens, ctx = (1, 130, 7, 64, 0, 300), (0, 0, 1000, 64, 10, 4097)
    kp, vp, table, seq, ks, vs = paged(P, lens, ctx, Hkv, D, P, layout)
    q = draw(3, sum(lens), Hq, D)
    out, lse, st = B.prompt_attention_paged(q, kp, vp, table, seq, cu(lens), kv_layout=layout, return_lse=True)
    assert int(st.item()) == 0
    o = 0
    for r, x in enumerate(lens):
        if x:
            check(out[o:o + x], lse[o:o + x], reference(q[o:o + x], ks[r], vs[r], D ** -0.5, True))
        o += x


def test_paged_is_packed_bit_for_bit(B):
    """The same keys from pages or packed: the same blocks, so the same result."""
    lens, ctx = (700, 33), (0, 0)
    kp, vp, table, seq, ks, vs = paged(1, lens, ctx, 2, 128, 64, "HND")
    q = draw(4, sum(lens), 16, 128)
    a = B.prompt_attention_paged(q, kp, vp, table, seq, cu(lens), return_lse=True)
    b = B.prompt_attention(q, torch.cat(ks), torch.cat(vs), cu(lens), return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_chunks_make_the_whole(B):
    """A prompt in chunks over the growing cache is the whole prompt."""
    n, Hq, Hkv, D, P = 1111, 8, 2, 128, 32
    kp, vp, table, _, ks, vs = paged(9, (n,), (0,), Hkv, D, P, "NHD")
    q = draw(8, n, Hq, D)
    want = reference(q, ks[0], vs[0], D ** -0.5, True)
    o = 0
    for x in (500, 1, 127, 128, 355):
        seq = torch.tensor([o + x], dtype=torch.int32, device="cuda")
        out, lse, st = B.prompt_attention_paged(q[o:o + x], kp, vp, table, seq, cu([x]), kv_layout="NHD", return_lse=True)
        assert int(st.item()) == 0
        check(out, lse, [w[o:o + x] for w in want])
        o += x


def test_padded_batch_is_left_alone(B):
    """Rows before the first and behind the last sequence hold NaN in the inputs and keep their outputs."""
    lens, Hq, Hkv, D = (100, 31), 8, 2, 64
    q, k, v = (draw(s, 10 + 131 + 60, H, D) for s, H in ((1, Hq), (2, Hkv), (3, Hkv)))
    for x in (q, k, v):
        x[:10], x[141:] = math.nan, math.inf
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    o, l, st = B.prompt_attention(q, k, v, cu(lens, 10), out=out, lse=lse)
    assert int(st.item()) == 0 and o is out and l is lse
    assert (out[:10] == 7).all() and (out[141:] == 7).all() and (lse[:10] == 7).all() and (lse[141:] == 7).all()
    for a, b in ((10, 110), (110, 141)):
        check(out[a:b], lse[a:b], reference(q[a:b], k[a:b], v[a:b], D ** -0.5, True))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (2, 2, 64)])
def test_values_that_a_query_does_not_see(B, bad, Hq, Hkv, D):
    """A key or value that is not finite changes the queries that see it, and no other: not the earlier
    ones in its own block of keys, not the other sequences."""
    lens = (300, 77)
    n = sum(lens)
    q, k, v = draw(1, n, Hq, D), draw(2, n, Hkv, D), draw(3, n, Hkv, D)
    clean = B.prompt_attention(q, k, v, cu(lens), return_lse=True)
    for which, at in (("v", 40), ("v", 299), ("k", 201), ("v", 300)):
        x = {"k": k.clone(), "v": v.clone()}
        x[which][at, Hkv - 1, 5] = bad
        out, lse, st = B.prompt_attention(q, x["k"], x["v"], cu(lens), return_lse=True)
        assert int(st.item()) == 0
        o = 0
        for m in lens:
            want, wl = OR.attention(q[o:o + m], x["k"][o:o + m], x["v"][o:o + m], D ** -0.5)
            got, gl = out[o:o + m].double().cpu().numpy(), lse[o:o + m].double().cpu().numpy()
            rows = (np.arange(m) + o < at) if o <= at < o + m else np.ones(m, bool)
            ref = reference(q[o:o + m], k[o:o + m], v[o:o + m], D ** -0.5, True)
            check(out[o:o + m][torch.from_numpy(rows)], lse[o:o + m][torch.from_numpy(rows)],
                  [r[torch.from_numpy(rows)] for r in ref])
            if which == "v":  # those that see it: the same infinities and NaN in the same places, and the rest as it was
                assert (np.isnan(got) == np.isnan(want)).all() and (np.isinf(got) == np.isinf(want)).all()
                assert (gl - clean[1][o:o + m].double().cpu().numpy() == 0).all() or np.allclose(gl, wl, rtol=0, atol=1e-5)
            o += m


def test_paged_values_that_a_query_does_not_see(B):
    lens, ctx = (200,), (150,)
    for layout in ("HND", "NHD"):
        kp, vp, table, seq, ks, vs = paged(5, lens, ctx, 1, 128, 64, layout)
        q = draw(3, 200, 8, 128)
        clean, _, _ = B.prompt_attention_paged(q, kp, vp, table, seq, cu(lens), kv_layout=layout)
        page = int(table[0, 240 // 64])
        (vp[page, 0, 240 % 64] if layout == "HND" else vp[page, 240 % 64, 0])[9] = math.nan  # key 240: query 90
        out, _, st = B.prompt_attention_paged(q, kp, vp, table, seq, cu(lens), kv_layout=layout)
        assert int(st.item()) == 0
        check(out[:90], None, [r[:90] for r in reference(q, ks[0], vs[0], 128 ** -0.5, True)])
        assert torch.isnan(out[90:, :, 9]).all() and not torch.isnan(out[:, :, :9]).any()


def test_strides(B):
    """Heads and tokens apart, and a layout with the heads outermost."""
    n, Hq, Hkv, D = 200, 4, 2, 64
    q, k, v = (draw(s, 2 * n, H + 1, D + 8)[::2, 1:, :D] for s, H in ((1, Hq), (2, Hkv), (3, Hkv)))
    out, _, _ = B.prompt_attention(q, k, v, cu([n]))
    assert torch.equal(out, B.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu([n]))[0])
    t = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    assert torch.equal(out, B.prompt_attention(*t, cu([n]))[0])
    one = B.prompt_attention(q[:1], k[:1], v[:1], cu([1]))[0]
    assert torch.equal(one[0], v[0].repeat_interleave(2, 0))  # one key: its value, exactly


def test_bad_lengths_are_flagged(B):
    q, k, v = draw(1, 64, 4, 64), draw(2, 64, 2, 64), draw(3, 64, 2, 64)
    good = B.prompt_attention(q, k, v, cu([64]))[0]
    for bad in ([0, 40, 30, 64], [0, 64, 65], [-3, 64]):
        out, _, st = B.prompt_attention(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert int(st.item()) == B.DEV_STATUS["bad_seqlen"]
    _, _, st = B.prompt_attention(q, k, v, cu([64]), cu_seqlens_k=torch.tensor([0, 65], dtype=torch.int32, device="cuda"))
    assert int(st.item()) == B.DEV_STATUS["bad_seqlen"]
    kp, vp, table, seq, _, _ = paged(2, (64,), (0,), 2, 64, 16, "HND")
    for n in (63, 1000, -1):
        _, _, st = B.prompt_attention_paged(q, kp, vp, table, torch.full_like(seq, n), cu([64]))
        assert int(st.item()) == B.DEV_STATUS["bad_seqlen"]
    for p in (-1, kp.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = p
        _, _, st = B.prompt_attention_paged(q, kp, vp, t, seq, cu([64]))
        assert int(st.item()) == B.DEV_STATUS["bad_page"]
    assert torch.equal(good, B.prompt_attention(q, k, v, cu([64]))[0])


def test_repeated_runs_are_bit_identical(B):
    lens = (900, 1, 300, 64, 2000, 7)
    n = sum(lens)
    q, k, v = draw(1, n, 16, 128), draw(2, n, 2, 128), draw(3, n, 2, 128)
    first = B.prompt_attention(q, k, v, cu(lens), return_lse=True)
    for _ in range(10):
        again = B.prompt_attention(q, k, v, cu(lens), return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_streams_and_graphs(B):
    lens = torch.tensor([0, 300, 500], dtype=torch.int32, device="cuda")
    q, k, v = draw(1, 600, 8, 128), draw(2, 600, 1, 128), draw(3, 600, 1, 128)
    want = B.prompt_attention(q, k, v, lens)[0][:500]
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([B.prompt_attention(q, k, v, lens)[0] for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o[:500], want) for group in outs for o in group)
    out, st = torch.zeros_like(q), B.new_status("cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.prompt_attention(q, k, v, lens, out=out, status=st)
    for new in ([0, 300, 500], [0, 1, 600], [0, 0, 77]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        e = new[-1]
        assert torch.equal(out[:e], B.prompt_attention(q, k, v, lens)[0][:e]) and not out[e:].any()


def test_cut_on_streams_and_in_a_graph(B):
    # 40 queries on 5000 keys of 2 kv heads are cut; each call has counters and scratch of its own.
    cq, ck = cu([40]), cu([5000])
    q, k, v = draw(1, 40, 8, 128), draw(2, 6000, 2, 128), draw(3, 6000, 2, 128)
    want = B.prompt_attention(q, k, v, cq, cu_seqlens_k=ck)[0]
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs += [B.prompt_attention(q, k, v, cq, cu_seqlens_k=ck)[0] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out, other, st = torch.zeros_like(q), torch.zeros_like(q), B.new_status("cuda")
    graphs = []
    for o in (out, other):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            B.prompt_attention(q, k, v, cq, cu_seqlens_k=ck, out=o, status=st)
    for n, m in ((40, 5000), (40, 6000), (3, 2000), (40, 50), (40, 5000)):
        cq.copy_(cu([n]))
        ck.copy_(cu([m]))
        for o in (out, other):
            o.zero_()
        for g in (*graphs, graphs[0]):
            g.replay()
        torch.cuda.synchronize()
        want = B.prompt_attention(q, k, v, cq, cu_seqlens_k=ck)[0]
        for o in (out, other):
            assert torch.equal(o[:n], want[:n]) and not o[n:].any()
    assert int(st.item()) == 0


@pytest.mark.parametrize("batch", [385, 3000])
def test_a_large_batch_of_short_prompts(B, batch):
    # Lengths 0 to 4, here and there 70: every sequence by itself is the same sequence.
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 5, (batch,), generator=g)
    lens[::97] = 70
    n = int(lens.sum())
    q, k, v = draw(1, n, 8, 64), draw(2, n, 4, 64), draw(3, n, 4, 64)
    out, lse, st = B.prompt_attention(q, k, v, cu(lens.tolist()), return_lse=True)
    assert int(st.item()) == 0
    at = [0, *lens.cumsum(0).tolist()]
    for r in (0, 1, 2, 96, 97, 98, 383, 384, batch - 2, batch - 1):
        a, b = at[r], at[r + 1]
        one, one_lse, _ = B.prompt_attention(q[a:b], k[a:b], v[a:b], cu([b - a]), return_lse=True)
        assert torch.equal(out[a:b], one) and torch.equal(lse[a:b], one_lse), r
    # every row is written: the whole against one call per hundred sequences
    for r in range(0, batch, 100):
        a, b = at[r], at[min(r + 100, batch)]
        part, _, _ = B.prompt_attention(q[a:b], k[a:b], v[a:b], cu(lens[r:r + 100].tolist()))
        assert torch.equal(out[a:b], part), r


def test_lengths_that_overlap_leave_no_row_out(B):
    # The descending boundaries are flagged; the three sequences between them are the same rows.
    q, k, v = draw(1, 512, 2, 64), draw(2, 512, 1, 64), draw(3, 512, 1, 64)
    want = B.prompt_attention(q, k, v, cu([512]))[0]
    bad = torch.tensor([0, 512, 0, 512, 0, 512], dtype=torch.int32, device="cuda")
    out, _, st = B.prompt_attention(q, k, v, bad)
    assert int(st.item()) == B.DEV_STATUS["bad_seqlen"] and torch.equal(out, want)


def test_refusals(B):
    q, k, v, c = draw(1, 8, 8, 64), draw(2, 8, 2, 64), draw(3, 8, 2, 64), cu([8])
    for args, kw, what in (((q.float(), k, v, c), {}, "dtype"), ((q, k, v[:4], c), {}, "agree"),
                           ((q[:, :6], k, v, c), {}, "1, 2, 4 or 8"), ((q[:, :5], k, v, c), {}, "num_heads"),
                           ((q, k[:4], v[:4], c), {}, "cu_seqlens_k"), ((q, k, v, c.long()), {}, "cu_seqlens"),
                           ((q, k, v, c), dict(sm_scale=0.0), "sm_scale"), ((q, k, v, c), dict(sm_scale=math.nan), "sm_scale"),
                           ((q, k, v, c), dict(out=torch.empty(8, 8, 64, device="cuda")), "out"),
                           ((q, k, v, c), dict(lse=torch.empty(8, 4, device="cuda")), "lse"),
                           ((q[..., :32], k[..., :32], v[..., :32], c), {}, "head_dim"),
                           ((q.transpose(1, 2), k, v, c), {}, "contiguous"),
                           ((draw(1, 8, 8, 65)[..., 1:], k, v, c), {}, "align|multiples")):
        with pytest.raises(B.HpcError, match=what):
            B.prompt_attention(*args, **kw)
    kp, vp, table, seq, _, _ = paged(2, (8,), (0,), 2, 64, 16, "HND")
    for kw, what in ((dict(q=q[:, :, :32]), "head_dim"), (dict(table=table[:0]), "block_table"), (dict(kp=kp.float()), "dtype"),
                     (dict(lay="DNH"), "kv_layout")):
        with pytest.raises(B.HpcError, match=what):
            B.prompt_attention_paged(kw.get("q", q), kw.get("kp", kp), vp, kw.get("table", table), seq, c,
                                     kv_layout=kw.get("lay", "HND"))
    out, lse, st = B.prompt_attention(q[:0], k[:0], v[:0], cu([0]), return_lse=True)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8) and int(st.item()) == 0

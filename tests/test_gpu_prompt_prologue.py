"""The prompt prologue against the fp64 oracle.

Tolerances. The kernel normalises and rotates in fp32 (a relative error of a few 2^-24 of the pair's
larger element) and rounds once: bf16 results lie within half a bf16 step of the fp64 value plus that,
so within 2^-8 |y| (1 + 2^-8) + 2^-20 max|pair|. E4M3 codes may differ from the fp64 value's code only
where that value is within 1e-5 (relative) of the midpoint of two codes."""
import numpy as np
import pytest
import torch

from oracle import fp8 as OF
from oracle import prompt as OR

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def make(lens, ctx, Hq, Hkv, D, P, kv, layout, seed=0, pad=(0, 0)):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    rows = pad[0] + n + pad[1]
    qkv = torch.randn((rows, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16)
    cu = torch.tensor([pad[0] + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    total = [a + b for a, b in zip(lens, ctx)]
    need = [-(-t // P) for t in total]
    N = sum(need) + 2
    perm = torch.randperm(N, generator=g)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
    o = 0
    for r, h in enumerate(need):
        table[r, :h] = perm[o:o + h]
        o += h
    shape = (N, Hkv, P, D) if layout == "HND" else (N, P, Hkv, D)
    dt = torch.uint8 if kv == "e4m3" else torch.bfloat16
    pages = [torch.randint(0, 100, shape, generator=g).to(dt) for _ in range(2)]
    c = dict(qkv=qkv, cu=cu, seq_lens=torch.tensor(total, dtype=torch.int32), table=table, k=pages[0], v=pages[1],
             qw=1 + 0.2 * torch.randn(D, generator=g), kw=1 + 0.2 * torch.randn(D, generator=g))
    if kv == "e4m3":
        c["ks"], c["vs"] = 0.005 + 0.02 * torch.rand(Hkv, generator=g), 0.005 + 0.02 * torch.rand(Hkv, generator=g)
    return c


def run(B, c, Hq, Hkv, kv, layout, **kw):
    d = {k: t.cuda() for k, t in c.items()}
    q, k, st = B.prompt_prologue(d["qkv"], d["cu"], d["qw"], d["kw"], d["k"], d["v"], d["table"], d["seq_lens"], Hq, Hkv,
                                 kv_dtype=kv, kv_layout=layout, k_scale=d.get("ks"), v_scale=d.get("vs"), **kw)
    return d, q, k, int(st.item())


def near_bf16(got, want, pairs):
    """|got - want| within half a bf16 step and the fp32 arithmetic (see the module's docstring)."""
    D = want.shape[-1]
    big = np.maximum(np.abs(pairs[..., :D // 2]), np.abs(pairs[..., D // 2:]))
    tol = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) + 2.0 ** -20 * np.concatenate([big, big], -1) + 1e-30
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


@pytest.mark.parametrize("lens,ctx,Hq,Hkv,D,P,kv,layout", [
    ((1,), (0,), 1, 1, 64, 16, "bf16", "HND"),
    ((1, 7, 0, 33, 1), (0, 100, 5, 131000, 15), 8, 2, 64, 16, "bf16", "HND"),
    ((5, 130, 1, 64), (0, 0, 4095, 63), 16, 2, 128, 64, "bf16", "NHD"),
    ((40, 3), (0, 17), 3, 3, 128, 32, "e4m3", "HND"),
    ((70, 1, 19), (1, 0, 30000), 64, 8, 128, 128, "e4m3", "NHD"),
    ((20,), (0,), 6, 2, 64, 16, "e4m3", "HND"),
    (tuple([1, 2] * 600), tuple([3, 0] * 600), 4, 4, 64, 16, "bf16", "HND"),
])
def test_against_the_oracle(B, lens, ctx, Hq, Hkv, D, P, kv, layout):
    c = make(lens, ctx, Hq, Hkv, D, P, kv, layout, seed=sum(lens) + D)
    d, q, k, st = run(B, c, Hq, Hkv, kv, layout)
    assert st == 0
    wq, wk, wv, writes = OR.prologue(c["qkv"], c["cu"].tolist(), c["seq_lens"].tolist(), c["qw"], c["kw"], 1e-6, 1e6,
                                     Hq, Hkv, P, c["table"].tolist())
    near_bf16(q.double().cpu().numpy(), wq, wq)
    near_bf16(k.double().cpu().numpy(), wk, wk)
    for name, want, scale in (("k", wk, c.get("ks")), ("v", wv, c.get("vs"))):
        pages, before = d[name].cpu(), c[name].clone()
        idx = torch.tensor([writes[i] for i in range(len(writes))])
        got = pages[idx[:, 0], :, idx[:, 1]] if layout == "HND" else pages[idx[:, 0], idx[:, 1]]
        if kv == "bf16":
            near_bf16(got.double().numpy(), want, want)
            if name == "v":
                assert torch.equal(got, c["qkv"][:, Hq + Hkv:])
        else:
            y = want / scale.double().numpy()[None, :, None]
            codes = OF.encode_array(y)
            bad = (got.numpy() != codes) & ~(OF.midpoint_distance(y) <= 1e-5)
            assert not bad.any()
        # nothing else in the cache changed
        if layout == "HND":
            before[idx[:, 0], :, idx[:, 1]] = got
        else:
            before[idx[:, 0], idx[:, 1]] = got
        assert torch.equal(pages.view(torch.uint8), before.view(torch.uint8))


def test_one_token_prompts_are_the_decode_prologue(B):
    """A prompt of one token is a decode step's new token: same codes, q within a bf16 step."""
    Hq, Hkv, D, P = 16, 4, 128, 64
    lens, ctx = (1,) * 9, (0, 1, 63, 64, 65, 1000, 16383, 131071, 500)
    c = make(lens, ctx, Hq, Hkv, D, P, "e4m3", "HND", seed=4)
    d, q, _, st = run(B, c, Hq, Hkv, "e4m3", "HND")
    e = {k: t.cuda() for k, t in c.items()}
    q1 = B.prologue(e["qkv"], e["qw"], e["kw"], e["k"], e["v"], e["table"], e["seq_lens"], Hq, Hkv, kv_dtype="e4m3",
                    k_scale=e["ks"], v_scale=e["vs"])
    assert st == 0
    assert (q.float() - q1.float()).abs().max() <= 2.0 ** -7 * q1.float().abs().max()
    diff = (d["k"].int() - e["k"].int()).abs()
    assert int(diff.max()) <= 1 and int((diff > 0).sum()) <= 4  # codes at a midpoint of two
    assert torch.equal(d["v"], e["v"])


def test_values_of_every_size_into_an_e4m3_cache(B):
    """V is only divided by its scale: against the quotient in fp32, infinities, NaN, overflow and small scales included."""
    n, Hkv, D, P = 512, 2, 128, 64
    g = torch.Generator().manual_seed(11)
    bits = torch.randint(0, 65536, (n, 3 * Hkv, D), generator=g, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    near = torch.randn((n, 3 * Hkv, D), generator=g).to(torch.bfloat16)
    c = make((n,), (0,), Hkv, Hkv, D, P, "e4m3", "NHD", seed=2)
    for x in (bits, near):
        for vs in (torch.tensor([0.37, 3.1]), torch.tensor([1e-6, 2.0 ** -9]), torch.tensor([0.0117, 1e4])):
            c["qkv"], c["vs"] = x, vs
            d, _, _, st = run(B, c, Hkv, Hkv, "e4m3", "NHD")
            assert st == 0
            y = x[:, 2 * Hkv:].float() / vs[:, None]
            got = d["v"].cpu()[c["table"][0, :n // P].long()].reshape(n, Hkv, D)
            nan = y.isnan()
            assert torch.equal((got & 127) == 127, nan)
            codes = torch.from_numpy(OF.encode_array(y.double().nan_to_num(0).clamp(-448, 448).numpy()).astype(np.uint8))
            assert torch.equal(got[~nan], codes[~nan])


def test_padded_rows_are_left_alone(B):
    Hq, Hkv, D, P = 8, 2, 64, 16
    c = make((5, 9), (0, 3), Hq, Hkv, D, P, "bf16", "HND", pad=(2, 6))
    c["qkv"][:2], c["qkv"][-6:] = float("nan"), float("nan")
    q0 = torch.full((22, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k0 = torch.full((22, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    d, q, k, st = run(B, c, Hq, Hkv, "bf16", "HND", q_out=q0, k_out=k0)
    assert st == 0 and q is q0 and k is k0
    for t in (q, k):
        assert (t[:2] == 7).all() and (t[16:] == 7).all() and torch.isfinite(t).all() and not (t[2:16] == 7).all(-1).any()


def test_bad_lengths_and_pages_are_flagged(B):
    Hq, Hkv, D, P = 8, 2, 64, 16
    c = make((4, 4, 4, 4), (0, 0, 0, 0), Hq, Hkv, D, P, "bf16", "HND", seed=8)
    c["seq_lens"][0] = 3        # shorter than its new tokens
    c["seq_lens"][1] = 33       # beyond the table (2 pages)
    c["table"][2, 0] = 1000     # outside the pool
    d, q, k, st = run(B, c, Hq, Hkv, "bf16", "HND")
    assert st == B.DEV_STATUS["bad_seqlen"] | B.DEV_STATUS["bad_page"]
    assert (q[:8] == 0).all() and (k[:8] == 0).all() and (q[8:] != 0).any(-1).all()
    changed = (d["k"].cpu() != c["k"]).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert changed == [int(c["table"][3, 0])]
    c["cu"] = torch.tensor([0, 12, 4, 12, 16], dtype=torch.int32)  # descends
    _, _, _, st = run(B, c, Hq, Hkv, "bf16", "HND")
    assert st & B.DEV_STATUS["bad_seqlen"]


def test_refusals(B):
    Hq, Hkv, D, P = 8, 2, 64, 16
    c = {k: t.cuda() for k, t in make((4,), (0,), Hq, Hkv, D, P, "bf16", "HND").items()}

    def call(**kw):
        a = {**c, **kw}
        return B.prompt_prologue(a["qkv"], a["cu"], a["qw"], a["kw"], a["k"], a["v"], a["table"], a["seq_lens"],
                                 a.get("Hq", Hq), Hkv, q_out=a.get("q_out"))

    for kw, what in ((dict(Hq=7), "qkv"), (dict(cu=c["cu"][:1]), "cu_seqlens"), (dict(cu=c["cu"].long()), "cu_seqlens"),
                     (dict(qw=c["qw"][:32]), "norm"), (dict(table=c["table"][:0]), "block_table"),
                     (dict(q_out=torch.empty((4, Hq, D), device="cuda")), "q_out"), (dict(k=c["k"].float()), "cache"),
                     (dict(qkv=c["qkv"].float()), "qkv")):
        with pytest.raises(B.HpcError, match=what):
            call(**kw)
    odd = torch.empty(4 * (Hq + 2 * Hkv) * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, Hq + 2 * Hkv, D)
    with pytest.raises(B.HpcError, match="align"):
        call(qkv=odd)
    q, k, st = call(qkv=c["qkv"][:0], cu=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert q.shape[0] == 0 and int(st.item()) == 0

"""Cached tokens as packed rows, for equality: a bf16 value is copied, an E4M3 value is its code's value times the scale,
rounded once to fp32 (exact for a scale that is a power of two) and once to bf16, as here. And prompt attention over E4M3
caches by way of them, against fp64 attention over the values that the rows hold."""
import math

import pytest
import torch

from oracle import fp8 as OF
from tests.test_gpu_prompt_attention import check, cu, draw, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def cache(seed, lens, Hkv, D, P, layout, kv):
    """Random pages of random bytes (E4M3: no NaN code) in random order; rows in fp32 on the side, without the scale."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // P) for n in lens]
    N = sum(need) + 2
    shape = (N, P, Hkv, D)
    pages, rows = [], []
    values = torch.tensor([OF.e4m3_to_float(c) for c in range(256)], dtype=torch.float64).float()
    perm = torch.randperm(N, generator=g)
    table = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32)
    o = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[o:o + n]
        o += n
    for _ in range(2):
        if kv == "e4m3":
            x = torch.randint(0, 256, shape, generator=g, dtype=torch.int32)
            x[(x & 127) == 127] = 0
            f, x = values[x.long()], x.to(torch.uint8)
        else:
            x = torch.randn(shape, generator=g).to(torch.bfloat16)
            f = x.float()
        rows.append([torch.cat([f[p] for p in table[r, :need[r]]] or [f[:0].reshape(0, Hkv, D)])[:n] for r, n in enumerate(lens)])
        pages.append((x.transpose(1, 2).contiguous() if layout == "HND" else x).cuda())
    scales = [0.01 + torch.rand(Hkv, generator=g) for _ in range(2)] if kv == "e4m3" else (None, None)
    want = []
    for f, s in zip(rows, scales):
        f = torch.cat(f) if f else None
        want.append((f if s is None else f * s[:, None]).to(torch.bfloat16).cuda())
    kw = dict(kv_dtype=kv, kv_layout=layout)
    if kv == "e4m3":
        kw.update(k_scale=scales[0].cuda(), v_scale=scales[1].cuda())
    return pages, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), want, kw


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Hkv,D,P,layout", [
    ((1,), 1, 64, 16, "HND"),
    ((0, 5, 0, 333, 64, 1), 8, 128, 16, "NHD"),
    ((100, 7, 2000), 3, 64, 1, "HND"),
    ((257, 4096), 2, 128, 48, "HND"),
    ((31, 9000, 2), 8, 128, 64, "NHD"),
    (tuple(range(40)) * 20, 1, 64, 7, "HND"),
])
def test_rows(B, kv, lens, Hkv, D, P, layout):
    (kp, vp), table, seq, (k, v), kw = cache(len(lens), lens, Hkv, D, P, layout, kv)
    n = sum(lens)
    for room in (n, n + 37):
        out = [torch.full((room, Hkv, D), -5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        ko, vo, c, st = B.gather_tokens(kp, vp, table, seq, room, k_out=out[0], v_out=out[1], **kw)
        assert int(st.item()) == 0 and c.tolist() == cu(lens).tolist()
        assert torch.equal(ko[:n], k) and torch.equal(vo[:n], v)
        assert (ko[n:] == -5).all() and (vo[n:] == -5).all()  # rows of no request


def test_special_codes(B):
    """Every E4M3 code, NaN and both zeros among them."""
    codes = torch.arange(256, dtype=torch.uint8).reshape(1, 1, 4, 64).cuda()
    one = torch.full((1,), 0.5, device="cuda")
    table, seq = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda")
    k, v, _, st = B.gather_tokens(codes, codes, table, seq, 4, kv_dtype="e4m3", k_scale=one, v_scale=one)
    want = torch.tensor([0.5 * OF.e4m3_to_float(c) for c in range(256)], dtype=torch.float64).to(torch.bfloat16)
    got = k.flatten().cpu()
    assert int(st.item()) == 0 and torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.view(torch.int16)[~got.isnan()], want.view(torch.int16)[~want.isnan()])
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))


def test_lengths_and_pages_that_do_not_fit(B):
    (kp, vp), table, seq, (k, v), kw = cache(3, (10, 20, 30, 5), 2, 64, 16, "HND", "bf16")
    ko, _, c, st = B.gather_tokens(kp, vp, table, seq, 31, k_out=torch.zeros(31, 2, 64, dtype=torch.bfloat16, device="cuda"))
    assert c.tolist() == [0, 10, 30, 30, 30] and int(st.item()) == B.DEV_STATUS["capacity"]
    assert torch.equal(ko[:30], k[:30]) and not ko[30:].any()
    _, _, c, st = B.gather_tokens(kp, vp, table, seq, 0)
    assert c.tolist() == [0] * 5 and int(st.item()) == B.DEV_STATUS["capacity"]
    for bad in (-1, 1000, 2 ** 31 - 1):
        odd = seq.clone()
        odd[1] = bad
        ko, _, c, st = B.gather_tokens(kp, vp, table, odd, 65)
        assert c.tolist() == [0, 10, 10, 40, 45] and int(st.item()) == B.DEV_STATUS["bad_seqlen"]
        assert torch.equal(ko[10:45], k[30:])
    for bad in (-1, kp.shape[0], 2 ** 31 - 1):
        odd = table.clone()
        odd[2, 1] = bad
        ko, vo, c, st = B.gather_tokens(kp, vp, odd, seq, 65)
        assert int(st.item()) == B.DEV_STATUS["bad_page"]
        assert not ko[46:60].any() and not vo[46:60].any() and torch.equal(ko[:46], k[:46]) and torch.equal(ko[60:], k[60:])
    big = torch.full((3,), 48, dtype=torch.int32, device="cuda")  # sums past the capacity, time and again
    _, _, c, st = B.gather_tokens(kp, vp, table[:3], big, 100)
    assert c.tolist() == [0, 48, 96, 96]


@pytest.mark.parametrize("kv,P,layout,D", [("e4m3", 16, "NHD", 128), ("e4m3", 64, "HND", 64), ("bf16", 48, "HND", 128),
                                           ("e4m3", 5, "HND", 128)])
def test_prompt_attention_by_way_of_rows(B, kv, P, layout, D):
    lens, total, Hq, Hkv = (1, 130, 7, 300), (1, 130, 1007, 2300), 8, 2
    (kp, vp), table, seq, (k, v), kw = cache(P, total, Hkv, D, P, layout, "bf16")
    if kv == "e4m3":  # values of the size that keys have
        scale = torch.tensor([0.02, 0.05], device="cuda")
        shape = (-1, 1, 1) if layout == "HND" else (-1, 1)
        kp, vp = [(x.float() / scale.view(shape)).to(torch.float8_e4m3fn) for x in (kp, vp)]
        kw = dict(kv_dtype="e4m3", kv_layout=layout, k_scale=scale, v_scale=scale)
        k, v, _, _ = B.gather_tokens(kp, vp, table, seq, sum(total), **kw)
        back = (kp.float() * scale.view(shape)).to(torch.bfloat16)
        if layout == "HND":
            back = back.transpose(1, 2)
        assert torch.equal(k[1:131], torch.cat([back[p] for p in table[1] if p >= 0])[:130])
    q = draw(3, sum(lens), Hq, D)
    out, lse, st = B.prompt_attention_paged(q, kp, vp, table, seq, cu(lens), return_lse=True, kv_tokens=sum(total) + 3, **kw)
    assert int(st.item()) == 0
    o = p = 0
    for x, m in zip(lens, total):
        check(out[o:o + x], lse[o:o + x], reference(q[o:o + x], k[p:p + m], v[p:p + m], D ** -0.5, True))
        o, p = o + x, p + m
    # a bound that the last request does not fit: it sees no keys
    out, lse, st = B.prompt_attention_paged(q, kp, vp, table, seq, cu(lens), return_lse=True, kv_tokens=2000, **kw)
    assert int(st.item()) == B.DEV_STATUS["capacity"] and not out[138:].any() and (lse[138:] == -math.inf).all()


def test_a_chunk_into_an_e4m3_cache(B):
    """The prologue writes a chunk of a prompt behind a cached prefix, and the chunk attends to all of it."""
    n, before, Hq, Hkv, D, P = 70, 150, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    kp, vp = torch.zeros((2, 20, P, Hkv, D), dtype=torch.uint8, device="cuda")
    table = torch.randperm(20, generator=torch.Generator().manual_seed(2)).to(torch.int32).reshape(1, 20).cuda()
    kw = dict(kv_dtype="e4m3", kv_layout="NHD", k_scale=torch.tensor([0.03, 0.05], device="cuda"),
              v_scale=torch.tensor([0.02, 0.01], device="cuda"))
    w = torch.ones(D, device="cuda")
    for m, x in ((before, before), (before + n, n)):
        qkv = torch.randn((x, Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        seq = torch.tensor([m], dtype=torch.int32, device="cuda")
        q, k_new, _ = B.prompt_prologue(qkv, cu([x]), w, w, kp, vp, table, seq, Hq, Hkv, **kw)
    out, lse, st = B.prompt_attention_paged(q, kp, vp, table, seq, cu([n]), return_lse=True, kv_tokens=before + n, **kw)
    assert int(st.item()) == 0
    k, v, _, _ = B.gather_tokens(kp, vp, table, seq, before + n, **kw)
    # A code is off by half a step at most: 2^-4 of the value, or 2^-10 scales below 2^-6 scales. The row and k_new are
    # rounded to bf16, 2^-8 each. No value reaches 448 scales: a normalised row's are at most sqrt(128) in size.
    err = (k[before:].double() - k_new.double()).abs()
    scale = kw["k_scale"].double()[:, None]
    assert (err <= k_new.double().abs() * (2.0 ** -4 + 2.0 ** -7) + scale * 2.0 ** -10).all()
    check(out, lse, reference(q, k, v, D ** -0.5, True))


def test_streams_and_graphs(B):
    (kp, vp), table, seq, (k, v), kw = cache(9, (300, 0, 41), 2, 128, 16, "HND", "e4m3")
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs += [B.gather_tokens(kp, vp, table, seq, 341, **kw) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], k) and torch.equal(o[1], v) for o in outs)
    q, c, st = draw(1, 50, 4, 128), cu([9, 0, 41]), B.new_status("cuda")
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.prompt_attention_paged(q, kp, vp, table, seq, c, kv_tokens=341, out=out, status=st, **kw)
    for lens in ((300, 0, 41), (9, 5, 41), (200, 16, 48)):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        table[1, 0] = 0
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, B.prompt_attention_paged(q, kp, vp, table, seq, c, kv_tokens=341, **kw)[0]), lens
    assert int(st.item()) == 0


def test_refusals(B):
    (kp, vp), table, seq, _, kw = cache(1, (5, 9), 2, 64, 16, "HND", "e4m3")
    q, c = draw(1, 4, 4, 64), cu([1, 3])
    for call, what in ((lambda: B.gather_tokens(kp, vp, table, seq, 14), "dtype"),
                       (lambda: B.gather_tokens(kp, vp, table, seq, 14, kv_dtype="e4m3"), "k_scale"),
                       (lambda: B.gather_tokens(kp, vp, table[:1], seq, 14, **kw), "block_table"),
                       (lambda: B.gather_tokens(kp, vp[1:], table, seq, 14, **kw), "differ"),
                       (lambda: B.gather_tokens(kp, vp, table, seq.long(), 14, **kw), "seq_lens"),
                       (lambda: B.gather_tokens(kp, vp, table, seq, -1, **kw), "kv_tokens"),
                       (lambda: B.gather_tokens(kp, vp, table, seq, 14, k_out=q, **kw), "k_out"),
                       (lambda: B.prompt_attention_paged(q, kp, vp, table, seq, c, kv_dtype="e4m3"), "kv_tokens"),
                       (lambda: B.prompt_attention_paged(q, kp, vp, table, seq, c), "dtype")):
        with pytest.raises(B.HpcError, match=what):
            call()

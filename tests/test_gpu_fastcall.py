"""The short way into the library gives what the long way gives, takes the calls it should take, and leaves the
others to it."""
import pytest
import torch

from tests.test_gpu_prompt_attention import cu, draw, paged
from tests.test_gpu_prompt_prologue import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    assert binding._fast is not None, "_fastcall.so is not built"
    return binding


class Spy:
    """Counts the calls that the fast module takes (a result) and leaves (None)."""

    def __init__(self, module):
        self.module, self.taken, self.left = module, 0, 0

    def __getattr__(self, name):
        f = getattr(self.module, name)

        def call(*a):
            r = f(*a)
            if r is None:
                self.left += 1
            else:
                self.taken += 1
            return r
        return call


def both(B, monkeypatch, f, taken=True):
    """f() the short way and the long way."""
    spy = Spy(B._fast)
    with monkeypatch.context() as m:
        m.setattr(B, "_fast", spy)
        a = f()
    assert (spy.taken > 0 and spy.left == 0) if taken else spy.taken == 0
    with monkeypatch.context() as m:
        m.setattr(B, "_fast", None)
        b = f()
    return a, b


def equal(a, b):
    a = list(a.__dict__.values()) if hasattr(a, "__dataclass_fields__") else a
    b = list(b.__dict__.values()) if hasattr(b, "__dataclass_fields__") else b
    for x, y in zip(a, b, strict=True):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.shape == y.shape and x.dtype == y.dtype and x.device == y.device
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_prompts(B, monkeypatch):
    q, k, v, c = draw(1, 90, 8, 64), draw(2, 90, 2, 64), draw(3, 90, 2, 64), cu([40, 50])
    for kw in ({}, dict(return_lse=True), dict(causal=False, sm_scale=0.3), dict(cu_seqlens_k=cu([60, 30]))):
        equal(*both(B, monkeypatch, lambda: B.prompt_attention(q, k, v, c, **kw)))
    wide = torch.cat([q, k, v], 1)
    equal(*both(B, monkeypatch, lambda: B.prompt_attention(wide[:, :8], wide[:, 8:10], wide[:, 10:], c)))
    kp, vp, table, seq, _, _ = paged(1, (40, 50), (3, 70), 2, 64, 16, "NHD")
    equal(*both(B, monkeypatch, lambda: B.prompt_attention_paged(q, kp, vp, table, seq, c, kv_layout="NHD", return_lse=True)))
    for kv, layout in (("bf16", "HND"), ("e4m3", "NHD")):
        d = {n: t.cuda() for n, t in make((4, 9), (0, 20), 8, 2, 128, 16, kv, layout).items()}
        equal(*both(B, monkeypatch, lambda: B.prompt_prologue(
            d["qkv"], d["cu"], d["qw"], d["kw"], d["k"], d["v"], d["table"], d["seq_lens"], 8, 2, kv_dtype=kv,
            kv_layout=layout, k_scale=d.get("ks"), v_scale=d.get("vs"))))


def test_verify(B, monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(0)
    p = torch.softmax(torch.randn(3, 4, 50, generator=g, device="cuda"), -1)
    x = torch.randint(0, 50, (3, 3), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(3, 4, generator=g, device="cuda")
    n = torch.tensor([3, 1, 0], dtype=torch.int32, device="cuda")
    q = p[:, :3].contiguous()
    for kw in ({}, dict(draft_lens=n), dict(seq_lens=n + 9, draft_lens=n)):
        equal(*both(B, monkeypatch, lambda: B.verify_drafts(x, p, q, u, **kw)))
        equal(*both(B, monkeypatch, lambda: B.verify_drafts(x, p.bfloat16(), None, u, **kw)))
    # padded rows go the long way
    equal(*both(B, monkeypatch, lambda: B.verify_drafts(x, p[:, :, :49], q[:, :, :49], u), taken=False))


def test_pages(B, monkeypatch):
    table = torch.tensor([[3, 0, -1], [1, -1, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 5], dtype=torch.int32, device="cuda")
    ref = torch.tensor([1, 1, 0, 1, 0, 0], dtype=torch.int32, device="cuda")
    par = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")

    def filled(up):  # what lies past the listed moves is not part of the result
        up.moves[int(up.n_moves):] = 0
        return up

    equal(*both(B, monkeypatch, lambda: filled(B.resize_pages(table, lens, lens + 20, ref, 16))))
    equal(*both(B, monkeypatch, lambda: filled(B.fork_pages(table, lens, ref, par, 16))))
    equal(*both(B, monkeypatch, lambda: filled(B.compact_pages(table, ref))))
    moves = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")

    def copy():
        c = [torch.arange(96, dtype=torch.uint8, device="cuda").view(6, 16) for _ in range(3)]
        return [B.copy_pages(c, moves, one), *c]
    equal(*both(B, monkeypatch, copy))


def test_refused_calls_go_the_long_way(B, monkeypatch):
    q, k, v, c = draw(1, 9, 8, 64), draw(2, 9, 2, 64), draw(3, 9, 2, 64), cu([9])
    for args in ((q, k, v[:4], c), (q.float(), k, v, c), (q.cpu(), k, v, c), (None, k, v, c), (q, k, v, c.long()),
                 (q[:, :6], k, v, c), ([1], k, v, c)):
        spy = Spy(B._fast)
        with monkeypatch.context() as m:
            m.setattr(B, "_fast", spy)
            with pytest.raises((B.HpcError, AttributeError)):
                B.prompt_attention(*args)
        assert spy.taken == 0 and spy.left == 1


def test_status_words_are_apart_and_captures_make_their_own(B):
    q, k, v, c = draw(1, 9, 8, 64), draw(2, 9, 2, 64), draw(3, 9, 2, 64), cu([9])
    words = [B.prompt_attention(q, k, v, c)[2] for _ in range(300)]
    assert len({w.data_ptr() for w in words}) == 300
    assert all(w.shape == (1,) and w.dtype == torch.int32 for w in words) and not any(int(w) for w in words[::37])
    bad = torch.tensor([0, 99], dtype=torch.int32, device="cuda")
    assert int(B.prompt_attention(q, k, v, bad)[2]) == B.DEV_STATUS["bad_seqlen"]
    assert int(B.prompt_attention(q, k, v, c)[2]) == 0
    cut = bad.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _, st = B.prompt_attention(q, k, v, cut)
    g.replay()
    assert int(st) == B.DEV_STATUS["bad_seqlen"]
    cut.copy_(c)
    g.replay()
    assert int(st) == 0  # zeroed at every replay
    assert torch.equal(out, B.prompt_attention(q, k, v, c)[0])

"""The serving operators together, as a serving loop runs them: prompts enter a paged cache, a prompt is
forked into samples, drafted tokens are written, attended to and verified, rejected ones are rolled back, the
pool is compacted, and decoding goes on. The state is followed on the side as plain per-row lists of keys
and values, and every attention result is compared with fp64 attention over them.

Tolerances: bf16 outputs of prompt attention as in test_gpu_prompt_attention; the decode steps within the
2e-3 of the decode tests."""
import math

import numpy as np
import pytest
import torch

from oracle import pages as OP
from oracle import verify as OV
from tests.helpers import BF16_TOL
from tests.test_gpu_prompt_attention import check, cu, reference

pytestmark = pytest.mark.gpu

HQ, HKV, D, P, N, M = 16, 2, 128, 16, 96, 16


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


class Loop:
    """A cache, its table, lengths and counts on the device, and the rows' keys and values on the side."""

    def __init__(self, B, layout, rows):
        self.B, self.layout = B, layout
        shape = (N, HKV, P, D) if layout == "HND" else (N, P, HKV, D)
        self.k = torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.table = torch.full((rows, M), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(N, dtype=torch.int32, device="cuda")
        self.w = [1 + 0.1 * torch.randn(D, device="cuda") for _ in range(2)]
        self.rows = [(torch.empty(0, HKV, D, dtype=torch.bfloat16, device="cuda"),) * 2 for _ in range(rows)]
        self.status = B.new_status("cuda")
        self.g = torch.Generator(device="cuda").manual_seed(5)

    def finish(self, up):
        self.B.copy_pages([self.k, self.v], up.moves, up.n_moves, status=self.status)
        self.table, self.ref = up.block_table, up.ref_count
        assert int(up.status.item()) == 0 and int(self.status.item()) == 0
        assert np.array_equal(self.ref.cpu().numpy(), OP.counts(self.table.tolist(), self.lens.tolist(), N, P))

    def resize(self, new):
        new = torch.as_tensor(new, dtype=torch.int32, device="cuda")
        up = self.B.resize_pages(self.table, self.lens, new, self.ref, P)
        self.lens = new
        self.finish(up)
        self.rows = [(k[:n], v[:n]) for (k, v), n in zip(self.rows, new.tolist())]

    def fork(self, parents):
        par = torch.tensor(parents, dtype=torch.int32, device="cuda")
        up = self.B.fork_pages(self.table, self.lens, self.ref, par, P)
        self.lens = up.seq_lens
        self.finish(up)
        self.rows = [self.rows[f] for f in parents]

    def compact(self):
        self.finish(self.B.compact_pages(self.table, self.ref))
        n = int((self.ref > 0).sum())
        assert int(self.table.max()) == n - 1

    def write(self, new):
        """`new` tokens of each row through the prompt prologue, into slots that the lengths already count.
        Returns the queries, packed."""
        n = sum(new)
        qkv = torch.randn((n, HQ + 2 * HKV, D), generator=self.g, device="cuda").to(torch.bfloat16)
        c = cu(new)
        q, k, _ = self.B.prompt_prologue(qkv, c, *self.w, self.k, self.v, self.table, self.lens, HQ, HKV,
                                         kv_layout=self.layout, status=self.status)
        v = qkv[:, HQ + HKV:]
        o = 0
        for r, m in enumerate(new):
            kk, vv = self.rows[r]
            self.rows[r] = (torch.cat([kk, k[o:o + m]]), torch.cat([vv, v[o:o + m]]))
            o += m
        return q, k, v, c

    def attend(self, q, c, new):
        out, lse, _ = self.B.prompt_attention_paged(q, self.k, self.v, self.table, self.lens, c, kv_layout=self.layout,
                                                    return_lse=True, status=self.status)
        assert int(self.status.item()) == 0
        o = 0
        for r, m in enumerate(new):
            if m:
                check(out[o:o + m], lse[o:o + m], reference(q[o:o + m], *self.rows[r], D ** -0.5, True))
            o += m
        return out


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_serving_loop(B, layout):
    torch.manual_seed(1)
    s = Loop(B, layout, 3)
    # prompts, the third row still empty
    first = [37, 100, 0]
    s.resize(first)
    q, k, v, c = s.write(first)
    paged = s.attend(q, c, first)
    packed, _, st = B.prompt_attention(q, k, v, c)
    assert int(st.item()) == 0 and torch.equal(paged, packed)
    # a second chunk of the longer prompt
    s.resize([37, 141, 0])
    q, _, _, c = s.write([0, 41, 0])
    s.attend(q, c, [0, 41, 0])
    # three samples of the first prompt, one of the second
    s.fork([0, 0, 1, 0])
    rng = np.random.default_rng(3)
    V, T = 97, 2
    for step in range(4):
        # the last token and T drafted ones
        s.resize((s.lens + T + 1).tolist())
        q, _, _, c = s.write([T + 1] * 4)
        out = s.attend(q, c, [T + 1] * 4)
        multi, st, _ = B.decode_step_multi(q.view(4, T + 1, HQ, D), s.k, s.v, s.table, s.lens, HKV, 64, kv_layout=layout)
        assert int(st.item()) == 0
        for r in range(4):
            want = reference(q[(T + 1) * r:(T + 1) * (r + 1)], *s.rows[r], D ** -0.5, True)[0]
            assert float((multi[r].double() - want).abs().max()) <= BF16_TOL["max"]
        assert float((multi.flatten(0, 1) - out.float()).abs().max()) < 0.1
        # verification from given random numbers
        p = torch.softmax(2 * torch.randn(4, T + 1, V, generator=s.g, device="cuda"), -1)
        d = torch.softmax(torch.log(p[:, :T]) + 0.5 * torch.randn(4, T, V, generator=s.g, device="cuda"), -1)
        x = torch.multinomial(d.flatten(0, 1), 1, generator=s.g).view(4, T).to(torch.int32)
        u = torch.rand(4, T + 1, generator=s.g, device="cuda")
        tokens, acc, new_lens, st = B.verify_drafts(x, p, d, u, seq_lens=s.lens)
        assert int(st.item()) == 0
        for r in range(4):
            want, a = OV.verify_one(x[r].tolist(), p[r].double().cpu().numpy(), d[r].double().cpu().numpy(),
                                    u[r].tolist(), T)
            assert tokens[r].tolist() == want.tolist() and int(acc[r]) == a
        assert torch.equal(new_lens, s.lens - T + acc)
        # rejected tokens leave; sometimes a row ends or is drawn again from another
        s.resize(new_lens.tolist())
        if step == 1:
            s.fork([2, 1, 1, 3])
        if step == 2:
            s.compact()
    s.resize([0, int(s.lens[1]), 0, int(s.lens[3])])
    s.fork([1, 3])
    s.compact()
    # decoding goes on: one token by the decode prologue and the single-launch step
    s.resize((s.lens + 1).tolist())
    qkv = torch.randn((2, HQ + 2 * HKV, D), generator=s.g, device="cuda").to(torch.bfloat16)
    q = B.prologue(qkv, *s.w, s.k, s.v, s.table, s.lens, HQ, HKV, kv_layout=layout)
    out, st, _ = B.decode_step_fused(q, s.k, s.v, s.table, s.lens, HQ, HKV, 64, kv_layout=layout)
    assert int(st.item()) == 0
    # the new token's k through the prompt prologue, on copies of the cache
    _, k, _ = B.prompt_prologue(qkv, cu([1, 1]), *s.w, s.k.clone(), s.v.clone(), s.table, s.lens, HQ, HKV, kv_layout=layout)
    v = qkv[:, HQ + HKV:]
    for r in range(2):
        kk, vv = s.rows[r]
        want = reference(q[r:r + 1], torch.cat([kk, k[r:r + 1]]), torch.cat([vv, v[r:r + 1]]), D ** -0.5, True)[0]
        # k of the two prologues may differ by a bf16 step in single elements: 2^-8 of one key's weight
        assert float((out[r].double() - want[0]).abs().max()) <= BF16_TOL["max"] + 2e-3

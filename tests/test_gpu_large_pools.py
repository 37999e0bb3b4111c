"""Caches whose offsets pass 32 bits (2.6e9 elements each): what the pages around the decode step do at the far end of such a
pool is, byte for byte, what they do in a small one."""
import pytest
import torch

from tests.test_gpu_prompt_attention import cu, draw

pytestmark = pytest.mark.gpu

N, H, P, D = 40001, 8, 64, 128
LENS, TOTAL = (70, 1, 200), (200, 3000, 200)


@pytest.fixture(scope="module")
def B():
    from load_balanced_split_step_b200 import binding
    return binding


def pools(layout, dtype):
    """(small K, V and table, large K, V and table): the small pool's pages are the last of the large one's."""
    need = [-(-t // P) for t in TOTAL]
    n = sum(need)
    g = torch.Generator().manual_seed(3)
    ids = torch.randperm(n, generator=g).to(torch.int32)
    table = torch.full((len(TOTAL), max(need)), -1, dtype=torch.int32)
    o = 0
    for r, k in enumerate(need):
        table[r, :k] = ids[o:o + k]
        o += k
    shape = (H, P, D) if layout == "HND" else (P, H, D)
    dev = torch.Generator(device="cuda").manual_seed(4)
    small = [torch.randn((n, *shape), generator=dev, device="cuda").to(dtype) for _ in range(2)]
    large = []
    for s in small:
        big = torch.empty((N, *shape), dtype=dtype, device="cuda")
        big[N - n:] = s
        large.append(big)
    far = torch.where(table >= 0, table + (N - n), table)
    return small, table.cuda(), large, far.cuda(), n


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_prompts(B, layout):
    small, near, large, far, n = pools(layout, torch.bfloat16)
    seq, c = torch.tensor(TOTAL, dtype=torch.int32, device="cuda"), cu(LENS)
    qkv, w = draw(1, sum(LENS), 2 * H + 2 * H, D), torch.ones(D, device="cuda")
    got = []
    for (k, v), table in ((small, near), (large, far)):
        q, kn, st = B.prompt_prologue(qkv, c, w, w, k, v, table, seq, 2 * H, H, kv_layout=layout)
        out, lse, st2 = B.prompt_attention_paged(q, k, v, table, seq, c, kv_layout=layout, return_lse=True)
        rows = B.gather_tokens(k, v, table, seq, sum(TOTAL), kv_layout=layout)
        assert int(st.item()) == int(st2.item()) == int(rows[3].item()) == 0
        got.append((q, kn, out, lse, *rows[:3], k[len(k) - n:], v[len(v) - n:]))
    for a, b in zip(*got, strict=True):
        assert torch.equal(a, b)


def test_copies(B):
    _, _, (k, v), _, n = pools("HND", torch.bfloat16)
    moves = torch.tensor([[N - 1, 5], [N - n, N - n - 1], [N - 2, 33000]], dtype=torch.int32, device="cuda")
    st = B.copy_pages([k, v], moves, torch.tensor([3], dtype=torch.int32, device="cuda"))
    assert int(st.item()) == 0
    for t in (k, v):
        for a, b in moves.tolist():
            assert torch.equal(t[a], t[b])
